// pair_product.cuh -- the tensor-core matrix product inside the operators of a layer's
// training step: D[m, n] = sum_k A[m, k] B[n, k], two SMs to a tile.
//
// Operands are 16-bit planes (bfloat16, or binary16): a matrix of more precise values is
// the sum of its planes, and the product the sum of the plane products that matter (the
// terms), all in one accumulator.  Either operand may lie with k or with its rows
// contiguous (the tensor core reads both from shared memory), so no transpose is ever
// written.
//
// A cluster of two CTAs owns a tile of 256 rows of A and BN rows of B
// (tcgen05.mma.cta_group::2: each SM holds 128 rows of A, half of B's, and 128 x BN sums
// in its tensor memory), so a byte of B that one SM loads is used by two.  The grid is
// persistent.  In each CTA warp 0 loads (TMA, a ring of stages of 64 k, each with every
// plane), warp 1 of the first CTA issues the products of both, and eight warps take
// finished sums to the epilogue while the next tile's products run (two buffers of BN
// columns of tensor memory).  Products of one plane run at 1.91 PFLOP/s (8192 x 5120 x
// 34816, cuBLAS's measured burst is 1.96); stages of 128 k were no faster.
//
// With FOLD the sums of one stage (64 k, the small terms first) at a time are added up in
// registers: the tensor core's additions cut off instead of rounding, which over a whole
// row of f32 terms would cost more than the terms themselves keep.  The fold hides behind
// the products (1557 of 1536 cycles a stage of three terms); the epilogue, on the same
// warps, does not.
#pragma once

#include <cuda_fp16.h>

#include <algorithm>

#include "activation.cuh"
#include "oop_internal.cuh"
#include "rows.cuh"
#include "tc_ptx.cuh"

namespace oop {
namespace pair {

constexpr int kThreads = 384, kEpilogueWarps = 8;
constexpr int kTileM = 256, kDepth = 64, kMaxTerms = 6, kMaxStages = 8;
constexpr int kPlaneBytes = 128 * kDepth * 2;              // A's plane of a stage, in one CTA
constexpr int kHeader = 1024;                              // barriers, before the stages
constexpr int kOutBytes = 4096;                            // of each epilogue warp, behind the stages
constexpr int kSmem = 227 * 1024;

// Where finished sums go.
enum Epilogue {
    kPlain,      // beta * (alpha * sum), rounded once, to a matrix
    kGate,       // act(gate) * up, and the two themselves if they are kept
    kSplit       // alpha * sum + beta * C + diag on the diagonal, as two binary16 planes
};

struct Out {
    void *p0, *p1, *p2;            // matrix (p1: that of batch 1, or NULL); h, gate, up
    int64_t nb0, nb1, batch;       // bytes between rows of p0 (kSplit: of C), of p1 and p2; between batches of p0 (or C)
    float *slots;                  // where the parts' sums go
    const __half *c_hi, *c_lo;     // kSplit: C's planes, laid out as the result's
    const float *row_scale;        // kGate with FOLD: factors of the rows, and of the gates' and
    const float *col_scale[2];     // the ups' columns, powers of two
    float alpha, beta, diag;
    int planes;                    // kSplit: matrices of a plane
    int type, act;
    int wide;                      // 16-byte stores are allowed
};

// The tiles of a product.  Those from `whole` on are taken in parts of k, each an item of
// its own whose sums go to a slot of 256 x BN floats for another kernel to join: all tiles
// where they are few, else the last wave's where it would leave more than half of the SMs
// idle.
struct TileMap {
    int m_tiles, n_tiles, tiles;   // tiles of a batch
    int symmetric;                 // only tiles on and above the diagonal
    int whole, parts;
};

struct Job {
    CUtensorMap a, b[2];
    CUtensorMap a_turned, b_turned;   // a_half, b_half: the same matrix with its rows as k
    CUtensorMap result;               // kSplit: the planes, by blocks of 32 x 32
    Out out;
    int *status;
    int64_t M, N;                  // kGate: N features, BN / 2 of them to a tile
    TileMap map;
    int items;                     // of the map
    int k_blocks, segments;        // stages of a segment; with two, b[s] and a's plane + s * a_seg
    int planes_a, planes_b, terms;
    int a_plane, a_batch, a_seg, b_plane, b_batch;   // third coordinates
    int term_a[kMaxTerms], term_b[kMaxTerms];
    int stages, stage_bytes;
    int sum_blocks;                // stages of one sum in tensor memory
    int inject;                    // test hook: the first stage waits for 16 bytes that no copy brings
    int a_rows, b_rows;            // the operand lies with its rows contiguous
    int a_half, b_half;            // the operand is a result of that kind
    uint32_t idesc;
};

// ---- device ---------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_ctas() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// The shared address of a CTA's copy of a variable.
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t cta) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(ptx::smem_u32(p)), "r"(cta));
    return r;
}
// No memory is handed over with it (the tcgen05 fences order tensor memory), so the plain
// form does: releasing to the cluster costs about a thousand cycles.
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
// Arrives on the barrier at this offset in both CTAs once every product issued so far is done.
__device__ __forceinline__ void commit_both(const void *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            ptx::smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
// Shared-memory descriptor of a plane, 128-byte swizzle.  k contiguous: rows of 64 k,
// groups of 8 rows 1024 bytes apart.  Rows contiguous: blocks of 64 rows by 64 k, 8 KB
// each (the leading offset), in them one k every 128 bytes (groups of 8 k 1024 bytes
// apart).
__device__ __forceinline__ uint64_t plane_desc(uint32_t addr, int rows_contiguous) {
    uint64_t d = static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(rows_contiguous ? 8192 >> 4 : 1) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void load_sums(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 64 columns of this warp's 32 lanes added to sums held as pairs.
__device__ __forceinline__ void add_sums(uint32_t taddr, uint64_t *sums) {
    uint32_t r[64];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i)
        sums[i] = ptx::add2(sums[i], ptx::pack2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])));
}

// The same of 32 gates, and of the ups of their features 64 columns further on.
__device__ __forceinline__ void add_gates(uint32_t taddr, uint64_t *sums) {
    uint32_t r[64];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr), "r"(taddr + 64)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i)
        sums[i] = ptx::add2(sums[i], ptx::pack2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])));
}
// 32 sums from pair i on.
__device__ __forceinline__ void take_sums(const uint64_t *sums, float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) ptx::unpack2(sums[i], v[2 * i], v[2 * i + 1]);
}

// 32 columns of the warp's 32 rows (a lane's row each) to memory: `row` is the first
// one's, from column c on; `rows` and `cols` of them exist.  A lane's row goes through the
// warp's part of shared memory, so that a store covers whole 64- or 128-byte pieces of few
// rows instead of 16 bytes of 32 (the XOR keeps both sides free of bank conflicts).
template <int TYPE>
__device__ __forceinline__ void store_block(uint8_t *stage, const float (&v)[32], char *row, int64_t nb, int64_t rows,
                                            int64_t cols, int wide) {
    constexpr int kSize = plain_size(TYPE), E = 16 / kSize, kPieces = 32 / E;
    const int lane = threadIdx.x & 31;
    auto place = [&](int r, int piece) {
        return stage + r * (32 * kSize) + ((piece ^ (kPieces == 8 ? r & 7 : r >> 1 & 3)) * 16);
    };
    __syncwarp();                                          // the last block is out of the stage
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        float part[E];
#pragma unroll
        for (int i = 0; i < E; ++i) part[i] = v[k * E + i];
        Packed<TYPE, E> w;
        w.set(part);
        *reinterpret_cast<typename Words<16>::T *>(place(lane, k)) = w.raw;
    }
    __syncwarp();
    if (!wide) {                                           // a row at a time, a column to a lane
        using S = typename Plain<TYPE>::S;
        if (lane >= cols) return;
        const int most = static_cast<int>(rows < 32 ? rows : 32);
#pragma unroll 4
        for (int r = 0; r < most; ++r)
            reinterpret_cast<S *>(row + r * nb)[lane] = reinterpret_cast<const S *>(place(r, lane / E))[lane % E];
        return;
    }
    const int piece = lane % kPieces, first = lane / kPieces;
    uint4 w[kPieces];                                      // all of them before the first store, which the compiler could not pass
#pragma unroll
    for (int i = 0; i < kPieces; ++i) w[i] = *reinterpret_cast<const uint4 *>(place(i * (32 / kPieces) + first, piece));
    if (piece * E < cols) {                                // cols is a multiple of E
        char *p = row + first * nb + piece * 16;
        const int64_t step = nb * (32 / kPieces);
#pragma unroll
        for (int i = 0; i < kPieces; ++i, p += step)
            if (i * (32 / kPieces) + first < rows) *reinterpret_cast<uint4 *>(p) = w[i];
    }
}
__device__ __forceinline__ void store_block(int type, uint8_t *stage, const float (&v)[32], char *row, int64_t nb, int64_t rows,
                                            int64_t cols, int wide) {
    if (type == OOP_TYPE_F32) store_block<OOP_TYPE_F32>(stage, v, row, nb, rows, cols, wide);
    else if (type == OOP_TYPE_F16) store_block<OOP_TYPE_F16>(stage, v, row, nb, rows, cols, wide);
    else store_block<OOP_TYPE_BF16>(stage, v, row, nb, rows, cols, wide);
}

struct Tile {
    int m, n, z;                   // z: batch
    int part, parts;               // of k
    int slot;                      // of the part's sums; -1: a whole tile
};

// Item i: batches outermost, then bands of eight row tiles, so that the tiles of a wave
// share their operands in L2.
__device__ __forceinline__ Tile tile_of(const TileMap &j, int i) {
    Tile t;
    t.part = 0;
    t.parts = 1;
    t.slot = -1;
    if (i >= j.whole) {
        t.slot = i - j.whole;
        t.part = t.slot % j.parts;
        t.parts = j.parts;
        i = j.whole + t.slot / j.parts;
    }
    t.z = i / j.tiles;
    i -= t.z * j.tiles;
    if (j.symmetric) {                                     // row tile m has n_tiles - m tiles
        t.m = 0;
        for (int left = j.n_tiles; i >= left; --left) {
            i -= left;
            ++t.m;
        }
        t.n = t.m + i;
        return t;
    }
    const int band = i / (8 * j.n_tiles), rest = i - band * 8 * j.n_tiles;
    const int rows = min(8, j.m_tiles - 8 * band);
    t.n = rest / rows;
    t.m = 8 * band + rest - t.n * rows;
    return t;
}

// First stage of a tile's part of k (end: of the next one).
__device__ __forceinline__ int first_stage(const Job &j, const Tile &t) {
    return static_cast<int>(static_cast<int64_t>(j.k_blocks) * j.segments * t.part / t.parts);
}
__device__ __forceinline__ int end_stage(const Job &j, const Tile &t) {
    return static_cast<int>(static_cast<int64_t>(j.k_blocks) * j.segments * (t.part + 1) / t.parts);
}

// Whether a symmetric matrix of which only the tiles on and above the diagonal exist has
// to be read as its transpose at k of row tile `tile`: then the tensor core takes the
// mirrored tile with its rows contiguous, and nothing is ever mirrored in memory.
__device__ __forceinline__ int below(int half, int k, int tile) { return half && k / kTileM < tile; }

// 32 columns (from c) of the warp's rows (from r0) as two binary16 planes, each staged in
// its half of the warp's shared memory (swizzled as TMA reads it: 64-byte rows) and copied
// from there while the warp goes on: every tile of a wave ends at once, and plain stores
// held the products up for as long as L2 took to swallow them all (32 x 768 x 2048: 290 of
// 1840 us).
__device__ __forceinline__ void store_split(uint8_t *stage, const CUtensorMap *map, const Out &o, float (&v)[32], int z, int64_t r0,
                                            int64_t c, int64_t M) {
    const int lane = threadIdx.x & 31;
    if (o.c_hi) {
        const int64_t at = z * o.batch / 2 + (r0 + lane) * (o.nb0 / 2) + c;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            uint4 a = make_uint4(0, 0, 0, 0), b = a;
            if (r0 + lane < M && c + i < o.nb0 / 2) {      // whole pitches are readable
                a = *reinterpret_cast<const uint4 *>(o.c_hi + at + i);
                b = *reinterpret_cast<const uint4 *>(o.c_lo + at + i);
            }
            __half ha[8], hb[8];
            __builtin_memcpy(ha, &a, 16);
            __builtin_memcpy(hb, &b, 16);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[i + j] = fmaf(o.alpha, v[i + j], o.beta * (__half2float(ha[j]) + __half2float(hb[j])));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= o.alpha;
    }
    if (c == r0) {                                         // the diagonal crosses this block
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] += i == lane ? o.diag : 0.f;
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        uint8_t *part = stage + p * 2048;
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");    // the copy before the last has left this half
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            __half2 h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[i] = __floats2half2_rn(v[8 * k + 2 * i], v[8 * k + 2 * i + 1]);
                const float2 f = __half22float2(h[i]);
                v[8 * k + 2 * i] -= f.x;
                v[8 * k + 2 * i + 1] -= f.y;
            }
            uint4 w;
            __builtin_memcpy(&w, h, 16);
            *reinterpret_cast<uint4 *>(part + lane * 64 + ((k ^ (lane >> 1 & 3)) * 16)) = w;
        }
        ptx::fence_async_shared();
        __syncwarp();
        if (lane == 0) {
            asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                             reinterpret_cast<uint64_t>(map)),
                         "r"(ptx::smem_u32(part)), "r"(static_cast<int>(c)), "r"(static_cast<int>(r0)), "r"(z + p * o.planes)
                         : "memory");
            ptx::bulk_commit();
        }
    }
}

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], sums_full[4], sums_empty[4];
    uint32_t tmem;
    int abort;
};

template <int EPI, bool FOLD, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ Job j) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    constexpr int kPlaneB = BN / 2 * kDepth * 2;
    // Buffers of sums in tensor memory.  With FOLD a buffer is taken every 64 k, so four small ones
    // hide the way from the tensor core to the registers and back better than two; a tile of 256
    // columns then fills two of them, from the halves of each CTA's rows of B.
    constexpr int kBufCols = FOLD ? 128 : BN, kBuffers = FOLD ? 4 : 2, kHalves = BN / kBufCols;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            ptx::mbar_init(&sh.full[i], 1);
            ptx::mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < kBuffers; ++i) {
            ptx::mbar_init(&sh.sums_full[i], 1);
            ptx::mbar_init(&sh.sums_empty[i], 2 * kEpilogueWarps);
        }
        sh.abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_u32(&sh.tmem)),
                     "r"(static_cast<uint32_t>(kBuffers * kBufCols))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    ptx::tc_fence_before();
    __syncthreads();
    cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&sh.tmem);
    // all of the above may run while the kernel before this one ends
    let_next_start();
    wait_previous();
    const uint32_t stage0 = ptx::smem_u32(smem) + kHeader;
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1, total = j.items;
    // one second, and two microseconds for every product that a wait may be for
    const uint64_t limit = 1000000000ull + 2000ull * static_cast<uint64_t>(j.sum_blocks) * j.terms * 4;
    bool timed_out = false;
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = ptx::globaltimer();
        for (uint32_t it = 1;; ++it) {
            if (ptx::mbar_try_wait(bar, parity)) return true;
            if ((it & 3) == 0) {
                if (*const_cast<volatile int *>(&sh.abort)) return false;
                if (ptx::globaltimer() - t0 > limit) {
                    *const_cast<volatile int *>(&sh.abort) = 1;
                    timed_out = true;
                    return false;
                }
            }
        }
    };

    // With FOLD the epilogue's warps need more registers than an even share: the first warpgroup
    // gives up its own (128 * 48 + 256 * 224 of the 384 * 168 at launch).
    if (warp < 4) {
        if constexpr (FOLD) ptx::setmaxnreg_dec<48>();
        if (warp == 0 && ptx::elect_one()) {
            ptx::prefetch_tmap(&j.a);
            ptx::prefetch_tmap(&j.b[0]);
            ptx::prefetch_tmap(&j.b[1]);
            int stage = 0;
            uint32_t phase = 0;
            for (int i = first; i < total; i += step) {
                const Tile t = tile_of(j.map, i);
                const int am = t.m * kTileM + static_cast<int>(rank) * 128;
                const int bn = EPI == kGate ? t.n * (BN / 2) : t.n * BN + static_cast<int>(rank) * (BN / 2);
                bool ok = true;
                const int end = end_stage(j, t);
                for (int kb = first_stage(j, t); kb < end && ok; ++kb) {
                    ok = wait(&sh.empty[stage], phase ^ 1);
                    if (!ok) break;
                    const uint32_t bar = cluster_addr(&sh.full[stage], 0);
                    if (rank == 0) ptx::mbar_arrive_expect_tx(&sh.full[stage], 2 * j.stage_bytes + (i + kb == 0 ? j.inject * 16 : 0));
                    const int seg = kb >= j.k_blocks ? 1 : 0;
                    const int k = (kb - seg * j.k_blocks) * kDepth;
                    const bool a_turned = below(j.a_half, k, t.m), b_turned = below(j.b_half, k, t.n);
                    uint32_t dst = stage0 + stage * j.stage_bytes;
                    for (int p = 0; p < j.planes_a; ++p, dst += kPlaneBytes) {
                        const int z = p * j.a_plane + t.z * j.a_batch + seg * j.a_seg;
                        if (j.a_rows || a_turned) {
                            const CUtensorMap *am_map = a_turned ? &j.a_turned : &j.a;
                            load_3d(dst, am_map, bar, am, k, z);
                            load_3d(dst + 8192, am_map, bar, am + 64, k, z);
                        } else {
                            load_3d(dst, &j.a, bar, k, am, z);
                        }
                    }
                    const CUtensorMap *bm = b_turned ? &j.b_turned : &j.b[EPI == kGate ? rank : seg];
                    for (int p = 0; p < j.planes_b; ++p, dst += kPlaneB) {
                        const int z = p * j.b_plane + t.z * j.b_batch;
                        if (j.b_rows || b_turned) {
#pragma unroll
                            for (int c = 0; c < BN / 128; ++c) load_3d(dst + 8192 * c, bm, bar, bn + 64 * c, k, z);
                        } else {
                            load_3d(dst, bm, bar, k, bn, z);
                        }
                    }
                    if (++stage == j.stages) stage = 0, phase ^= 1;
                }
                if (!ok) break;
            }
            // the last stages are read before this CTA may end
            for (int i = 0; i < j.stages; ++i) {
                if (!wait(&sh.empty[stage], phase ^ 1)) break;
                if (++stage == j.stages) stage = 0, phase ^= 1;
            }
        }
        if (warp == 1 && rank == 0 && ptx::elect_one()) {
            int stage = 0, buf = 0;
            uint32_t phase = 0, buf_phase = 0;
            bool ok = true;
            for (int i = first; i < total && ok; i += step) {
                const Tile t = tile_of(j.map, i);
                const int end = end_stage(j, t);
                if constexpr (FOLD) {
                    for (int kb = first_stage(j, t); kb < end && ok; ++kb) {
                        ok = wait(&sh.full[stage], phase);
                        const uint32_t sa = stage0 + stage * j.stage_bytes, sb = sa + j.planes_a * kPlaneBytes;
                        const int a_rows = j.a_rows | below(j.a_half, kb * kDepth, t.m);
                        const int b_rows = j.b_rows | below(j.b_half, kb * kDepth, t.n);
                        const uint64_t ka = a_rows ? 128 : 2, kb_step = b_rows ? 128 : 2;      // 16 k, in 16-byte units
                        const uint32_t idesc = j.idesc | static_cast<uint32_t>(a_rows) << 15 | static_cast<uint32_t>(b_rows) << 16;
                        for (int h = 0; h < kHalves && ok; ++h) {
                            ok = wait(&sh.sums_empty[buf], buf_phase ^ 1);
                            if (!ok) break;
                            ptx::tc_fence_after();
                            uint32_t add = 0;
                            for (int q = 0; q < j.terms; ++q) {
                                const uint64_t da = plane_desc(sa + j.term_a[q] * kPlaneBytes, a_rows);
                                const uint64_t db = plane_desc(sb + j.term_b[q] * kPlaneB + h * 8192, b_rows);
#pragma unroll
                                for (int k = 0; k < kDepth / 16; ++k) {
                                    mma(tmem + buf * kBufCols, da + k * ka, db + k * kb_step, idesc, add);
                                    add = 1;
                                }
                            }
                            commit_both(&sh.sums_full[buf]);
                            if (++buf == kBuffers) buf = 0, buf_phase ^= 1;
                        }
                        if (!ok) break;
                        commit_both(&sh.empty[stage]);
                        if (++stage == j.stages) stage = 0, phase ^= 1;
                    }
                } else {                                   // a_half, b_half: not in this form
                    const uint64_t ka = j.a_rows ? 128 : 2, kb_step = j.b_rows ? 128 : 2;
                    const uint32_t idesc = j.idesc | static_cast<uint32_t>(j.a_rows) << 15 | static_cast<uint32_t>(j.b_rows) << 16;
                    ok = wait(&sh.sums_empty[buf], buf_phase ^ 1);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    uint32_t add = 0;
                    for (int kb = first_stage(j, t); kb < end; ++kb) {
                        ok = wait(&sh.full[stage], phase);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        const uint32_t sa = stage0 + stage * j.stage_bytes, sb = sa + j.planes_a * kPlaneBytes;
                        for (int q = 0; q < j.terms; ++q) {
                            const uint64_t da = plane_desc(sa + j.term_a[q] * kPlaneBytes, j.a_rows);
                            const uint64_t db = plane_desc(sb + j.term_b[q] * kPlaneB, j.b_rows);
#pragma unroll
                            for (int k = 0; k < kDepth / 16; ++k) {
                                mma(tmem + buf * kBufCols, da + k * ka, db + k * kb_step, idesc, add);
                                add = 1;
                            }
                        }
                        commit_both(&sh.empty[stage]);
                        if (++stage == j.stages) stage = 0, phase ^= 1;
                    }
                    if (!ok) break;
                    commit_both(&sh.sums_full[buf]);
                    if (++buf == kBuffers) buf = 0, buf_phase ^= 1;
                }
            }
        }
        __syncwarp();
    } else {
        if constexpr (FOLD) ptx::setmaxnreg_inc<224>();
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t empty_bar = cluster_addr(&sh.sums_empty[0], 0);
        uint8_t *stage_out = smem + kHeader + j.stages * j.stage_bytes + (warp - 4) * kOutBytes;
        const int element = plain_size(j.out.type);
        int buf = 0;
        uint32_t buf_phase = 0;
        constexpr int kCols = BN / 2;                      // of this warp
        bool ok = true;
        auto sums_ready = [&] {
            ok = __all_sync(0xffffffffu, wait(&sh.sums_full[buf], buf_phase));
            if (ok) ptx::tc_fence_after();
            return ok;
        };
        auto sums_taken = [&] {
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(empty_bar + 8 * buf);
            if (++buf == kBuffers) buf = 0, buf_phase ^= 1;
        };
        // The code from here to the stores is kept short: a tile runs it once, and unrolled for a
        // whole row and every type it took 28 us to be fetched, twice a small call's products.
        for (int i = first; i < total && ok; i += step) {
            const Tile t = tile_of(j.map, i);
            const int64_t r0 = static_cast<int64_t>(t.m) * kTileM + rank * 128 + quarter * 32, rows = j.M - r0;
            // a gate's pieces: the gates and ups of 32 features
            auto gate = [&](float (&g)[32], float (&u)[32], int64_t f) {
                if (rows <= 0 || f >= j.N) return;
                if constexpr (FOLD) {
                    const float by = lane < rows ? j.out.row_scale[r0 + lane] : 0.f;
                    const int64_t c = min(f + lane, j.N - 1);
                    const float of_g = j.out.col_scale[0][c], of_u = j.out.col_scale[1][c];
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const float bg = __shfl_sync(0xffffffffu, of_g, k), bu = __shfl_sync(0xffffffffu, of_u, k);
                        g[k] = g[k] * fminf(by, bg) * fmaxf(by, bg);       // the small one first: no step leaves fp32's
                        u[k] = u[k] * fminf(by, bu) * fmaxf(by, bu);       // range that the result does not leave
                    }
                }
                auto put = [&](const float (&v)[32], void *p, int64_t nb) {
                    store_block(j.out.type, stage_out, v, static_cast<char *>(p) + r0 * nb + f * element, nb, rows, j.N - f, j.out.wide);
                };
                if (j.out.p1) {
                    put(g, j.out.p1, j.out.nb1);
                    put(u, j.out.p2, j.out.nb1);
                }
                if constexpr (FOLD) {
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        const float4 h = activation_call(j.out.act, make_float4(g[k], g[k + 1], g[k + 2], g[k + 3]));
                        g[k] = h.x * u[k];
                        g[k + 1] = h.y * u[k + 1];
                        g[k + 2] = h.z * u[k + 2];
                        g[k + 3] = h.w * u[k + 3];
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) g[k] = activation_of(j.out.act, g[k]) * u[k];
                }
                put(g, j.out.p0, j.out.nb0);
            };
            auto plain = [&](float (&v)[32], int64_t c) {
                if (rows <= 0 || c >= j.N) return;
                if (t.slot >= 0) {
                    if constexpr (EPI == kSplit) {
                        if (lane == 0) ptx::bulk_wait_read();                  // the last tile's copies have left the stage
                        __syncwarp();
                    }
                    const int r = rank * 128 + quarter * 32, at = static_cast<int>(c - static_cast<int64_t>(t.n) * BN);
                    char *slot = reinterpret_cast<char *>(j.out.slots + (static_cast<int64_t>(t.slot) * kTileM + r) * BN + at);
                    store_block<OOP_TYPE_F32>(stage_out, v, slot, BN * 4, 32, 32, 1);
                } else if constexpr (EPI == kSplit) {
                    store_split(stage_out, &j.result, j.out, v, t.z, r0, c, j.M);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] *= j.out.alpha, v[k] *= j.out.beta;
                    char *base = j.out.p1 && t.z ? static_cast<char *>(j.out.p1) : static_cast<char *>(j.out.p0) + t.z * j.out.batch;
                    store_block(j.out.type, stage_out, v, base + r0 * j.out.nb0 + c * element, j.out.nb0, rows, j.N - c, j.out.wide);
                }
            };
            if constexpr (FOLD) {
                uint64_t sums[kCols / 2];                  // of each half: 64 columns, or 32 gates and 32 ups
#pragma unroll
                for (int c = 0; c < kCols / 2; ++c) sums[c] = 0;
                for (int kb = first_stage(j, t); kb < end_stage(j, t) && ok; ++kb) {
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) {
                        if (!sums_ready()) break;
                        const uint32_t from = tmem + lanes + buf * kBufCols;
                        if constexpr (EPI == kGate) add_gates(from + half * 32, sums + 32 * h);
                        else add_sums(from + half * 64, sums + 32 * h);
                        sums_taken();
                    }
                }
                if (!ok) break;
#pragma unroll
                for (int p = 0; p < kCols / 32; ++p) {
                    float v[32], u[32];
                    take_sums(sums + 16 * p, v);
                    if constexpr (EPI == kGate) {
                        if (p & 1) continue;
                        take_sums(sums + 16 * p + 16, u);
                        gate(v, u, static_cast<int64_t>(t.n) * (BN / 2) + p * 32 + half * 32);
                    } else {
                        plain(v, static_cast<int64_t>(t.n) * BN + half * kCols + p * 32);
                    }
                }
            } else {
                if (!sums_ready()) break;
                const uint32_t from = tmem + lanes + buf * kBufCols;
                if constexpr (EPI == kGate) {
                    const int at = half * (BN / 4);
#pragma unroll 1
                    for (int p = 0; p < BN / 4; p += 32) {
                        float g[32], u[32];
                        load_sums(from + at + p, g);
                        load_sums(from + BN / 2 + at + p, u);
                        if (p + 32 == BN / 4) sums_taken();
                        gate(g, u, static_cast<int64_t>(t.n) * (BN / 2) + at + p);
                    }
                } else {
#pragma unroll 1
                    for (int p = 0; p < kCols; p += 32) {
                        float v[32];
                        load_sums(from + half * kCols + p, v);
                        if (p + 32 == kCols) sums_taken();
                        plain(v, static_cast<int64_t>(t.n) * BN + half * kCols + p);
                    }
                }
            }
        }
        __syncwarp();
        if (EPI == kSplit && lane == 0) ptx::bulk_wait();
    }
    if (timed_out) record_status(j.status, OOP_ERR_DEVICE_TIMEOUT);
    __syncthreads();
    if (sh.abort) {                                        // copies and products in flight end before the CTA does
        const uint64_t t0 = ptx::globaltimer();
        while (ptx::globaltimer() - t0 < 50000000ull) __nanosleep(1000);
    }
    ptx::tc_fence_before();
    cluster_sync();
    ptx::tc_fence_after();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(static_cast<uint32_t>(kBuffers * kBufCols))
                     : "memory");
}

// use(z, row, column, sum of the parts in their order) for every element of the tiles in
// parts, four of a row at a time; a CTA of 256 threads to four rows (blockIdx.x =
// kJoinCtas * tile + rows).
constexpr int kJoinCtas = kTileM / 4;

template <int BN, class F>
__device__ __forceinline__ void each_joined(const TileMap &map, const float *slots, F &&use) {
    const Tile t = tile_of(map, map.whole + static_cast<int>(blockIdx.x / kJoinCtas) * map.parts);
    const int i = threadIdx.x * 4;
    if (i >= 4 * BN) return;
    const int at = static_cast<int>(blockIdx.x % kJoinCtas) * 4 * BN + i;
    const float *p = slots + static_cast<int64_t>(t.slot) * kTileM * BN + at;
    float4 v = *reinterpret_cast<const float4 *>(p);
#pragma unroll 4
    for (int k = 1; k < map.parts; ++k) {
        const float4 w = *reinterpret_cast<const float4 *>(p + static_cast<int64_t>(k) * kTileM * BN);
        v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    }
    use(t.z, static_cast<int64_t>(t.m) * kTileM + at / BN, static_cast<int64_t>(t.n) * BN + at % BN, v);
}

// ---- host -----------------------------------------------------------------

// Elements of a plane's row, which starts on 16 bytes, and bytes of a part of a workspace.
inline int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }
inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

constexpr int64_t kPairs = 76;                             // of SMs: sizes can be asked for without a GPU

// The tiles of a product of so many stages and terms, and which of them go in parts of at
// least eight stages: where the stages that saves (0.27 us for each term) outweigh the
// join's launch (8 us) and the slots' traffic (0.1 us each).
inline TileMap tile_map(int64_t M, int64_t N, int64_t cols, int64_t stages, int terms, int64_t batches, bool symmetric, bool in_parts) {
    TileMap m = {};
    const int64_t mt = (M + kTileM - 1) / kTileM, nt = (N + cols - 1) / cols;
    m.m_tiles = static_cast<int>(mt);
    m.n_tiles = static_cast<int>(nt);
    m.tiles = static_cast<int>(symmetric ? nt * (nt + 1) / 2 : mt * nt);
    m.symmetric = symmetric;
    const int64_t all = m.tiles * batches, last = all % kPairs;
    m.whole = static_cast<int>(all);
    m.parts = 1;
    if (in_parts && last > 0 && 2 * last <= kPairs && stages >= 16) {
        const int64_t n = std::min<int64_t>({kPairs / last, stages / 8, 16});
        const double saved = 0.27 * terms * static_cast<double>(stages - (stages + n - 1) / n);
        if (saved > 8.0 + 0.1 * static_cast<double>(last * n)) m.whole = static_cast<int>(all - last), m.parts = static_cast<int>(n);
    }
    return m;
}
inline int64_t tiles_in_parts(const TileMap &m, int64_t batches) { return m.tiles * batches - m.whole; }
inline size_t slot_bytes(const TileMap &m, int64_t batches, int64_t cols) {
    return (static_cast<size_t>(tiles_in_parts(m, batches)) * m.parts * kTileM * cols * 4 + 255) / 256 * 256;
}

// One operand: `planes` planes of `batches` matrices of `rows` x `k`, their rows or their
// k contiguous.
struct Operand {
    const void *p;
    int64_t inner, outer, pitch_bytes;         // contiguous extent, the other one, bytes between its lines
    int64_t matrix_bytes, matrices;            // all planes and batches, one after the other
    bool rows_contiguous;
    bool half;                                 // binary16, else bfloat16
};

inline bool make_map(CUtensorMap *map, const Operand &o, int tile_rows, bool block = false) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(o.inner), static_cast<cuuint64_t>(o.outer),
                                static_cast<cuuint64_t>(o.matrices)};
    // a stride over a single line is not used, but has to be a multiple of 16
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(o.outer > 1 ? o.pitch_bytes : 16),
                                   static_cast<cuuint64_t>(o.matrices > 1 ? o.matrix_bytes : 16)};
    const cuuint32_t box[3] = {block ? 32u : 64u, static_cast<cuuint32_t>(block ? 32 : o.rows_contiguous ? 64 : tile_rows), 1};
    const cuuint32_t ones[3] = {1, 1, 1};
    return fn(map, o.half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(o.p), dims,
              strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, block ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What the caller says of a product; the rest of the Job follows.
struct Spec {
    Operand a, b[2];
    int64_t M, N, K;               // K of one segment
    int batches, segments, planes_a, planes_b;
    bool in_parts;                 // out.slots is there for the tiles that go in parts
    int a_plane, a_batch, a_seg, b_plane, b_batch;
    bool symmetric;
    bool a_half, b_half;           // FOLD and 256 columns only
    Operand result;                // kSplit
    Out out;
};

// The terms that matter: planes i and j with i + j below the larger number of planes (each
// plane is 2^-8, or 2^-11, of the one before).
inline int list_terms(int pa, int pb, int (&ta)[kMaxTerms], int (&tb)[kMaxTerms]) {
    const int top = pa > pb ? pa : pb;
    int n = 0;
    for (int s = top - 1; s >= 0; --s)                     // small ones first
        for (int i = 0; i <= s; ++i)
            if (i < pa && s - i < pb) {
                ta[n] = i;
                tb[n++] = s - i;
            }
    return n;
}

inline int count_terms(int pa, int pb) {
    int ta[kMaxTerms], tb[kMaxTerms];
    return list_terms(pa, pb, ta, tb);
}

template <int EPI, bool FOLD, int BN>
cudaError_t launch(const Spec &s, int *status, cudaStream_t st) {
    Job j = {};
    if (!make_map(&j.a, s.a, 128) || !make_map(&j.b[0], s.b[0], BN / 2) || !make_map(&j.b[1], s.b[1], BN / 2))
        return cudaErrorInvalidValue;
    for (int i = 0; i < 2; ++i) {
        Operand o = i ? s.b[0] : s.a;
        o.rows_contiguous = true;
        if ((i ? s.b_half : s.a_half) && !make_map(i ? &j.b_turned : &j.a_turned, o, 0)) return cudaErrorInvalidValue;
    }
    if (EPI == kSplit && !make_map(&j.result, s.result, 0, true)) return cudaErrorInvalidValue;
    static_assert(BN == 256 || EPI != kSplit, "symmetric results have square tiles");
    j.a_half = s.a_half;
    j.b_half = s.b_half;
    j.out = s.out;
    j.status = status;
    j.M = s.M;
    j.N = s.N;
    constexpr int kTileN = EPI == kGate ? BN / 2 : BN;
    j.terms = list_terms(s.planes_a, s.planes_b, j.term_a, j.term_b);
    const int64_t blocks = (s.K + kDepth - 1) / kDepth;
    const int64_t most = (s.M + kTileM - 1) / kTileM * ((s.N + kTileN - 1) / kTileN) * s.batches;
    if (most * 16 > 0x7fffffffLL || blocks * s.segments > 0x7fffffffLL) return cudaErrorInvalidValue;
    j.map = tile_map(s.M, s.N, kTileN, blocks * s.segments, j.terms, s.batches, s.symmetric, s.in_parts);
    j.items = j.map.whole + static_cast<int>(tiles_in_parts(j.map, s.batches)) * j.map.parts;
    j.k_blocks = static_cast<int>(blocks);
    j.segments = s.segments;
    j.planes_a = s.planes_a;
    j.planes_b = s.planes_b;
    j.a_plane = s.a_plane, j.a_batch = s.a_batch, j.a_seg = s.a_seg, j.b_plane = s.b_plane, j.b_batch = s.b_batch;
    j.stage_bytes = s.planes_a * kPlaneBytes + s.planes_b * (BN / 2 * kDepth * 2);
    j.stages = (kSmem - kHeader - kEpilogueWarps * kOutBytes) / j.stage_bytes;
    if (j.stages > kMaxStages) j.stages = kMaxStages;
    j.inject = tc_take_inject();
    j.sum_blocks = FOLD ? 1 : static_cast<int>(blocks * s.segments);
    j.a_rows = s.a.rows_contiguous;
    j.b_rows = s.b[0].rows_contiguous;
    const uint32_t kind = s.a.half ? 0u : 1u;
    j.idesc = (1u << 4) | (kind << 7) | (kind << 10) | (static_cast<uint32_t>((FOLD ? 128 : BN) >> 3) << 17) |
              (static_cast<uint32_t>(kTileM >> 4) << 24);
    const int sms = device_sm_count();
    int64_t pairs = sms / 2 > 0 ? sms / 2 : 1;
    if (pairs > j.items) pairs = j.items;
    cudaError_t e = allow_smem<product_kernel<EPI, FOLD, BN>>();
    if (e != cudaSuccess) return e;
    if (FOLD) {                                            // another split would wait forever for its registers
        static const int registers = [] {
            cudaFuncAttributes attr = {};
            return cudaFuncGetAttributes(&attr, product_kernel<EPI, FOLD, BN>) == cudaSuccess ? attr.numRegs : 0;
        }();
        if (registers != 168) return cudaErrorLaunchOutOfResources;
    }
    const dim3 grid(static_cast<unsigned>(2 * pairs));
    const size_t smem = static_cast<size_t>(kHeader + j.stages * j.stage_bytes + kEpilogueWarps * kOutBytes);
    if (g_kernel_launches++ == 0) {                        // what comes before is not this library's to overlap with
        product_kernel<EPI, FOLD, BN><<<grid, kThreads, smem, st>>>(j);
        return cudaGetLastError();
    }
    return launch_dependent(product_kernel<EPI, FOLD, BN>, grid, kThreads, smem, st, j);
}

}  // namespace pair
}  // namespace oop
