// mxq_matmul.cu -- products of block-scaled FP8 operands on the tensor cores:
//   out[i, j] = sum_b 2^(sa(i, b) + sb(j, b)) sum_{k in block b} A[i, k] B[j, k]
// with blocks of 128 along the depth, accumulated in fp32.
//
// Every scale of this library is a power of two, so tcgen05.mma's block
// scaling (kind::mxf8f6f4, one UE8M0 byte per 32 elements of depth) applies
// it inside the instruction: the four 32-deep instructions of a 128-block name
// the same byte.  Tile scales (one per 128x128 weights) become that byte for
// 128 rows.  Nothing is rescaled in registers and the accumulator stays in
// tensor memory from the first block to the last.
//
// An operand's depth runs either along the rows in memory or across them
// (gradients); both are what one TMA box of 128 bytes x 128 and one matrix
// descriptor describe, so all three products of a linear layer are one kernel.
//
// One thread block (or a pair of them, on two SMs) is a pipeline of warps:
//   warp 0     TMA: boxes of both operands, 128 deep, into a ring of stages
//   warp 1     one thread issues scale copies and MMAs
//   warp 2, 3  gather the scale bytes of eight blocks (1024 of depth) of each operand
//   warps 4..  take finished sums out of tensor memory, round and store them
// Blocks walk over their tiles, so that loads and MMAs of the next tile run
// while the last one is being stored.
//
// What bounds it (GB300; the tensor cores' own time for a 256x256 tile and 128
// of depth is 497 clocks, 4.9 PFLOP/s at 2 GHz):
//   8192^3                       0.299 ms, 3.7 PFLOP/s, in six calls in a row,
//                                0.340 in 200: the board's power.  On operands
//                                of zeros 0.281 ms, 3.9 PFLOP/s.
//   rows of 7184 bytes           a box of 128 bytes lies across two 128-byte
//                                lines; the L2 serves five sectors for four:
//                                16384x4096x7184 2.7 PFLOP/s, at 8192 deep 3.6
//                                (in 200 calls 2.7 and 3.2).
//   few rows                     the weight's bytes: one token through
//                                8192x8192 15.1 us, 4.4 TB/s, of which 11 us
//                                are the stream at 6 TB/s and the rest the
//                                launch and the sum over a cluster; 48 tokens x 2 of 32 experts
//                                (4096x7184 each) at 5.6 TB/s of the weights that they chose.
//   experts with uneven loads    no unit: 16384 rows over 32 experts, 24 of
//                                which have fewer than 256, take 430 us, with the
//                                tensor pipes busy 48% of the time, the L2 46%
//                                and the HBM 35%.  An expert with few rows waits for
//                                its weight, one with many for the tensor cores,
//                                and their tiles come one expert after the other.
// A pair's stages take 32 KB a block of depth on each SM, which at the tensor
// cores' rate is 18 TB/s from the L2: wider sharing (clusters of four with
// multicast) would relieve it, but only 144 of the 152 SMs hold such clusters.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "mxq_device.cuh"
#include "mxq_layer.h"
#include "mxq_launch.cuh"
#include "mxq_tcgen05.cuh"

namespace mxq {
namespace {

constexpr int kMostExperts = 1024;
// Scales move in groups of two words a row, eight blocks of depth: a warp spends about 1000 clocks on a group (its loads,
// which the proxy fence waits for, the words' order and the fence), the tensor cores 4000 on its products.
constexpr int kGroup = 8;
constexpr int kRing = 2;  // groups, both in shared and in tensor memory

// The tensor core cuts off what a sum's 24 bits cannot hold instead of
// rounding it, so that the error of a long sum grows with its length: in one
// accumulation of normally distributed operands 2.2e-7 of the result's norm at
// a depth of 4096, 2.5e-7 at 4608 and 3e-6 at 33000, where a sum that is
// rounded has 1e-7 to 2e-7.  Operands of one sign have 1.4e-6 at 4096, those
// whose magnitudes spread over 2^20 along the depth 2.4e-6.  That is far below
// a bf16 result's own rounding (1.7e-3), but not below fp32's.  fp32 results
// deeper than 36 blocks are therefore summed in segments of about equal length
// (40 blocks at most), each added, rounded, to what the output holds, which
// keeps the error where it is at one segment's depth: 2.2e-7 at 8191, 2.8e-7 at
// 33000 (2.4e-6 and 2.9e-6 for the spread ones).  A segment more costs what its
// results' way to memory and back does (8192 x 4096 x 4096: 101 us, as bf16 in
// one segment 85).
constexpr int kSegment = 36;

// The operand whose rows are the accumulator's lanes is called P, the one
// whose rows are its columns Q.  Lanes come 128 at a time, columns in any
// multiple of 16.  Where tokens are few or an expert's, they are the columns:
// odd numbers of them then cost little more than their own products.  Where
// they are many they are the lanes, whose thread holds neighbours of one row
// of the output.
enum ScaleForm {
    kTiles,          // an fp32 power of two per 128x128 tile
    kAlongDepth,     // a byte per row and block, a row's bytes together
    kAcrossDepth,    // a byte per row and block, a block's bytes together
    kAcrossAligned,  // and those of four neighbouring rows in an aligned word
};

struct ScaleSource {
    const void* base;
    int64_t s_row, s_kb, s_expert;
    int64_t bytes;  // kAlongDepth: of the whole matrix
    int rows;
    int form;
};

enum RaggedBy { kNone, kRowsOfQ, kDepth };

struct Problem {
    ScaleSource sp, sq;
    const int32_t* offsets;
    void* out;
    int64_t ldo, out_expert;
    int E, depth;
    int p_rows, q_rows, p_tiles, q_tiles;
    int columns;  // of the accumulator a tile takes, where experts' rows do not decide it
    int segment;  // blocks of depth that one accumulation takes: see kSegment
    int whole;    // tiles in front of those that are taken in two halves (CG 2, kNone)
    int ragged;
    bool p_mn, q_mn;   // the operand's depth runs across its rows in memory
    bool p_expert;     // P is a stack of experts' weights
    bool out_bf16;
    bool wide;  // four neighbours of the output can be stored at once
};

struct Tile {
    int e, p0, q0, q_end;
    int columns;  // of the accumulator: q_end - q0, rounded up
    int kb0, kb1;
};

// Rows (or depth) of the experts: bound[e] .. bound[e + 1], and the tiles in front of expert e.
struct Ragged {
    int *bound, *tiles;
};

// Warp-wide: clamps the offsets into 0..limit and to be non-decreasing, and counts tiles of `step`.
__device__ void read_offsets(const Problem& g, int limit, int step, Ragged r) {
    const int lane = threadIdx.x & 31;
    int top = 0, sum = 0;
    for (int i0 = 0; i0 <= g.E; i0 += 32) {
        const int i = i0 + lane;
        int v = i <= g.E ? min(max(g.offsets[i], 0), limit) : 0;
        if (g.ragged == kDepth) v = min((v + 127) / 128 * 128, limit);
        v = max(v, top);
        for (int d = 1; d < 32; d *= 2) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, v, d);
            if (lane >= d) v = max(v, up);
        }
        const int prev_lane = __shfl_up_sync(0xFFFFFFFFu, v, 1);
        const int prev = lane ? prev_lane : top;
        int n = i > 0 && i <= g.E ? (v - prev + step - 1) / step : 0;
        for (int d = 1; d < 32; d *= 2) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, n, d);
            if (lane >= d) n += up;
        }
        if (i <= g.E) {
            r.bound[i] = v;
            r.tiles[i] = sum + n;
        }
        top = __shfl_sync(0xFFFFFFFFu, v, 31);
        sum += __shfl_sync(0xFFFFFFFFu, n, 31);
    }
}

// Tiles are numbered so that those in flight together share operands: groups
// of 16 tiles of P are walked along Q; within an expert the few tiles of its
// rows come first.
template <int PT, int QT>
__device__ __forceinline__ Tile tile_at(const Problem& g, const Ragged& r, int t) {
    Tile c;
    c.e = 0;
    c.kb0 = 0;
    c.kb1 = (g.depth + 127) >> 7;  // sizes are at most 2^30
    if (g.ragged == kRowsOfQ) {
        int lo = 0, hi = g.E - 1;  // the last expert whose tiles begin at or before t
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (r.tiles[mid] * g.p_tiles <= t)
                lo = mid;
            else
                hi = mid - 1;
        }
        c.e = lo;
        t -= r.tiles[lo] * g.p_tiles;
        const int n = r.tiles[lo + 1] - r.tiles[lo];
        c.q0 = r.bound[lo] + t % n * QT;
        c.q_end = min(r.bound[lo + 1], c.q0 + QT);
        c.columns = QT < 256 ? QT : (c.q_end - c.q0 + 15) & ~15;  // a narrow last tile loads less than two even ones
        c.p0 = t / n * PT;
        return c;
    }
    if (g.ragged == kDepth) {
        const int per = g.p_tiles * g.q_tiles;
        c.e = t / per;
        t -= c.e * per;
        c.kb0 = (r.bound[c.e] + 127) >> 7;  // only `depth` itself is no multiple of 128: nothing begins there
        c.kb1 = (r.bound[c.e + 1] + 127) >> 7;
    }
    // The last round's tiles come in halves of 128 columns where that fills it better.
    const int half = QT == 256 && g.ragged == kNone && t >= g.whole ? (t - g.whole) & 1 : -1;
    if (half >= 0) t = g.whole + ((t - g.whole) >> 1);
    constexpr int G = 16;  // 8192^3: 299 us; groups of eight 303, of four 309
    const int group = t / (G * g.q_tiles), first = group * G, n = min(G, g.p_tiles - first);
    t -= group * G * g.q_tiles;
    c.p0 = (first + t % n) * PT;
    c.q0 = t / n * g.columns;
    if (half > 0) c.q0 += 128;
    c.q_end = min(g.q_rows, c.q0 + (half >= 0 ? 128 : g.columns));
    c.columns = QT < 256 ? QT : min(g.columns, (c.q_end - c.q0 + 31) & ~31);
    if (c.q_end <= c.q0) {  // a half behind the last column: no work, and nothing to store
        c.q_end = c.q0;
        c.columns = 32;
        c.kb1 = c.kb0;
    }
    return c;
}

// The scales of W * 32 rows from row0 on and kGroup = 8 blocks from kb on, read
// by one warp.  Loads are unconditional, at indexes clamped into the operand:
// a row behind its end has no output and a block behind kb_end no product.
// They stay raw until pack(), so that all of a warp's loads are in flight at
// once, and those of the next group while the ring is full.
template <int W>
struct ScaleReader {
    uint32_t raw[8 * W];

    __device__ __forceinline__ void load(const ScaleSource& s, int e, int row0, int kb, int kb_end) {
        const int lane = threadIdx.x & 31;
        if (s.form == kTiles) {  // one of 8 blocks x W/4 tiles a lane
            const int tile = min((row0 >> 7) + min(lane >> 3, W / 4 - 1), (s.rows - 1) >> 7);
            raw[0] = static_cast<const uint32_t*>(
                s.base)[e * s.s_expert + tile * s.s_row + min(kb + (lane & 7), kb_end - 1) * s.s_kb];
            return;
        }
        const uint8_t* p = static_cast<const uint8_t*>(s.base);
        if (s.form == kAlongDepth) {  // eight bytes at any address: three words, shifted by pack()
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const int64_t at = min(row0 + 32 * i + lane, s.rows - 1) * s.s_row + kb;
                const uint8_t* word = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(p + at) & ~uintptr_t(3));
                if (word >= p && word + 12 <= p + s.bytes) {
#pragma unroll
                    for (int j = 0; j < 3; ++j) raw[3 * i + j] = reinterpret_cast<const uint32_t*>(word)[j];
                } else {  // at the matrix's ends, byte by byte into the same places
                    const int shift = (int)(p + at - word);
                    raw[3 * i] = raw[3 * i + 1] = raw[3 * i + 2] = 0;
#pragma unroll
                    for (int j = 0; j < 11; ++j)
                        if (j >= shift && j < shift + 8 && kb + j - shift < kb_end)
                            raw[3 * i + j / 4] |= (uint32_t)word[j] << (8 * (j & 3));
                }
            }
        } else if (s.form == kAcrossAligned) {  // four rows, 4 lane .. 4 lane + 3 of each 128, a word
#pragma unroll
            for (int i = 0; i < W / 4; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    raw[8 * i + j] = *reinterpret_cast<const uint32_t*>(p + min(row0 + 128 * i + 4 * lane, s.rows - 4) +
                                                                        min(kb + j, kb_end - 1) * s.s_kb);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    raw[8 * i + j] = p[min(row0 + 32 * i + lane, s.rows - 1) + min(kb + j, kb_end - 1) * s.s_kb];
        }
    }

    // Writes the UE8M0 bytes where tcgen05.cp takes them: of four blocks and 128
    // rows 512 bytes, row r's four at 16 (r % 32) + 4 (r / 32); the second four
    // blocks `next` bytes on.
    __device__ __forceinline__ void pack(const ScaleSource& s, int row0, int kb, uint8_t* to, int next) const {
        const int lane = threadIdx.x & 31;
        if (s.form == kTiles) {
            // 2^c has the byte c + 127: the exponent field, and 0 for the subnormal 2^-127; all else is NaN
            const uint32_t t = raw[0];
            const uint32_t c = (t & 0x7FFFFFu) == 0u && t - 1u < 0x7F7FFFFFu ? t >> 23 : t == 0x00400000u ? 0u : 255u;
#pragma unroll
            for (int a = 0; a < W / 4; ++a)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t v = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) v |= __shfl_sync(0xFFFFFFFFu, c, 8 * a + 4 * h + j) << (8 * j);
                    *reinterpret_cast<uint4*>(to + h * next + 512 * a + 16 * lane) = make_uint4(v, v, v, v);
                }
        } else if (s.form == kAcrossAligned) {
#pragma unroll
            for (int a = 0; a < W / 4; ++a)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t* w = raw + 8 * a + 4 * h;  // block j's bytes of four rows -> row i's of four blocks
                    const uint32_t lo01 = prmt(w[0], w[1], 0x5140), hi01 = prmt(w[0], w[1], 0x7362),
                                   lo23 = prmt(w[2], w[3], 0x5140), hi23 = prmt(w[2], w[3], 0x7362);
                    const uint32_t row[4] = {prmt(lo01, lo23, 0x5410), prmt(lo01, lo23, 0x7632), prmt(hi01, hi23, 0x5410),
                                             prmt(hi01, hi23, 0x7632)};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint32_t*>(to + h * next + 512 * a + 16 * (4 * (lane & 7) + i) + 4 * (lane >> 3)) =
                            row[i];
                }
        } else {
            uint32_t w[2][W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                if (s.form == kAlongDepth) {
                    const int64_t at = min(row0 + 32 * i + lane, s.rows - 1) * s.s_row + kb;
                    const uint32_t shift = 8 * ((uint32_t)(reinterpret_cast<uintptr_t>(s.base) + at) & 3u);
                    w[0][i] = __funnelshift_r(raw[3 * i], raw[3 * i + 1], shift);
                    w[1][i] = __funnelshift_r(raw[3 * i + 1], raw[3 * i + 2], shift);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        w[h][i] = raw[8 * i + 4 * h] | raw[8 * i + 4 * h + 1] << 8 | raw[8 * i + 4 * h + 2] << 16 |
                                  raw[8 * i + 4 * h + 3] << 24;
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int a = 0; a < W / 4; ++a)
                    *reinterpret_cast<uint4*>(to + h * next + 512 * a + 16 * lane) =
                        make_uint4(w[h][4 * a], w[h][4 * a + 1], w[h][4 * a + 2], w[h][4 * a + 3]);
        }
    }
};

__device__ __forceinline__ uint32_t canonical(uint32_t u) { return (u & 0x7FFFFFFFu) > 0x7F800000u ? 0x7FC00000u : u; }

__device__ __forceinline__ void store_one(const Problem& g, int64_t at, uint32_t u) {
    u = canonical(u);
    if (g.out_bf16)
        static_cast<uint16_t*>(g.out)[at] = (uint16_t)bf16_rne(u);
    else
        static_cast<uint32_t*>(g.out)[at] = u;
}

// Four neighbours of one output row, the first `n` of them inside.
__device__ __forceinline__ void store_four(const Problem& g, int64_t at, int n, float4 v) {
    const uint32_t u[4] = {canonical(__float_as_uint(v.x)), canonical(__float_as_uint(v.y)), canonical(__float_as_uint(v.z)),
                           canonical(__float_as_uint(v.w))};
    if (g.wide && n >= 4) {  // at is a multiple of four then
        if (g.out_bf16)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.out) + at) =
                make_uint2(bf16_rne(u[0]) | bf16_rne(u[1]) << 16, bf16_rne(u[2]) | bf16_rne(u[3]) << 16);
        else
            *reinterpret_cast<uint4*>(static_cast<uint32_t*>(g.out) + at) = make_uint4(u[0], u[1], u[2], u[3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) store_one(g, at + i, u[i]);
}

// 128 bf16 values of a row of the output, the first `n` of them inside, by 16
// threads: 16 aligned bytes a store, wherever the row begins.
__device__ __forceinline__ void store_row(uint16_t* to, const uint16_t* from, int n, int part, bool aligned) {
    if (aligned && 8 * part + 8 <= n) {
        *reinterpret_cast<uint4*>(to + 8 * part) = *reinterpret_cast<const uint4*>(from + 8 * part);
        return;
    }
    const int skip = (int)(reinterpret_cast<uintptr_t>(to) & 15u) / 2;  // values of the first 16 bytes that are not the row's
    for (int f = 8 * part - skip; f < n; f += 128) {  // part 0 has the row's last few, too
        if (f >= 0 && f + 8 <= n) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = from[f + 2 * i] | (uint32_t)from[f + 2 * i + 1] << 16;
            *reinterpret_cast<uint4*>(to + f) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (f + i >= 0 && f + i < n) to[f + i] = from[f + i];
        }
    }
}

// Blocks to a segment: as even as whole groups allow.
__device__ __forceinline__ int even_segment(const Problem& g, int depth) {
    const int n = (depth + g.segment - 1) / g.segment;
    return n <= 1 ? g.segment : ((depth + n - 1) / n + kGroup - 1) / kGroup * kGroup;
}

// QT: columns of the accumulator, at most for CG 2, where each tile has a
// width of its own.  CG 2: a pair of blocks, 256 lanes, each loading half of a
// tile's rows of Q.  CG 1: 128 lanes.  SPLIT: the blocks of a cluster share a
// tile, each with a part of the depth, and add their sums through shared
// memory.  ROWS: the output's rows are the lanes (CG 2), else the columns.
template <int QT, int CG, bool SPLIT, bool ROWS>
struct Shape {
    static constexpr int kQRows = QT / CG;                           // rows of Q that a block loads
    static constexpr int kPBytes = 128 * 128, kQBytes = kQRows * 128;
    static constexpr int kStageBytes = kPBytes + kQBytes;
    static constexpr int kOutWarps = CG == 2 && !ROWS ? 8 : 4;  // that take results out
    static constexpr int kThreads = 128 + 32 * kOutWarps;
    static constexpr int kStages = CG == 2 ? (ROWS ? 6 : 5) : QT == 128 ? (SPLIT ? 3 : 6) : QT == 64 ? 4 : 5;
    static constexpr int kQAtoms = QT <= 128 ? 1 : QT / 128;         // 128 scales each
    static constexpr int kScaleBytes = 512 * (1 + kQAtoms);           // of four blocks
    static constexpr int kScaleColumns = 4 * (1 + kQAtoms);
    static constexpr int kScaleParts = kRing * (kGroup / 4);
    // Two accumulators (one where a block has one tile).  Two of 256 columns and the scales exceed the 512 columns, so
    // there the second begins 64 columns before the first one's end and the
    // shared ones are taken out first.
    static constexpr int kAcc1 = QT == 256 ? 192 : QT;
    static constexpr int kScaleAt = QT == 256 ? 448 : SPLIT ? QT : 2 * QT;
    static constexpr int kUsed = kScaleAt + kScaleParts * kScaleColumns;
    static constexpr int kColumns = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
    static constexpr int kPerSm = CG == 2 || (QT == 128 && !SPLIT) ? 1 : 2;  // shared and tensor memory have room for
    static constexpr int kOutBytes = CG == 2 && !ROWS ? 2 * 64 * 128 * 2 : 0;  // bf16 results on their way out
    static constexpr int kBox = CG == 2 ? 64 : QT;  // rows of Q in one copy
    static constexpr int kBarriers = 2 * kStages + 2 * kRing + 4 + 1;
    static size_t smem(int E) {
        return 1024 + (size_t)kStages * kStageBytes + (size_t)kScaleParts * kScaleBytes + kOutBytes + 8 * kBarriers + 16 +
               (E ? 8 * (size_t)(E + 1) : 0);
    }
};

template <int QT, int CG, bool SPLIT, bool ROWS>
__global__ void __launch_bounds__(Shape<QT, CG, SPLIT, ROWS>::kThreads, Shape<QT, CG, SPLIT, ROWS>::kPerSm)
    matmul_kernel(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map,
                  const __grid_constant__ Problem g, const uint32_t idesc, const int tile_count) {
    using S = Shape<QT, CG, SPLIT, ROWS>;
    constexpr int PT = 128 * CG;
    extern __shared__ uint8_t raw[];
    uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t* scales = stages + S::kStages * S::kStageBytes;
    [[maybe_unused]] uint16_t* outs = reinterpret_cast<uint16_t*>(scales + S::kScaleParts * S::kScaleBytes);  // [64][128]
    uint8_t* bars = scales + S::kScaleParts * S::kScaleBytes + S::kOutBytes;
    volatile int* gave_up = reinterpret_cast<volatile int*>(bars + 8 * S::kBarriers);
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(bars + 8 * S::kBarriers + 4);
    Ragged rag;
    rag.bound = reinterpret_cast<int*>(bars + 8 * S::kBarriers + 16);
    rag.tiles = rag.bound + g.E + 1;

    const uint32_t full = smem_u32(bars), empty = full + 8 * S::kStages, sc_full = empty + 8 * S::kStages,
                   sc_empty = sc_full + 8 * kRing, acc_full = sc_empty + 8 * kRing, acc_empty = acc_full + 16,
                   drained = acc_empty + 16;
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x / 32, 0), lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 || SPLIT ? cluster_rank() : 0;
    const uint32_t pair_rank = CG == 2 ? rank : 0;
    const bool leader = pair_rank == 0;

    if (warp == 0) {
        if (lane == 0) {
            prefetch_map(&p_map);
            prefetch_map(&q_map);
            for (int i = 0; i < S::kStages; ++i) {
                mbar_init(full + 8 * i, 1);
                mbar_init(empty + 8 * i, 1);
            }
            for (int i = 0; i < kRing; ++i) {
                mbar_init(sc_full + 8 * i, 2 * CG);
                mbar_init(sc_empty + 8 * i, 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(acc_full + 8 * i, 1);
                mbar_init(acc_empty + 8 * i, CG * S::kOutWarps);
            }
            mbar_init(drained, 1);
            *gave_up = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    } else if (warp == 1) {
        tmem_alloc<CG>(smem_u32(tmem_at), S::kColumns);
    }
    wait_for_stream();
    if (warp == 2 && g.ragged != kNone) read_offsets(g, g.ragged == kDepth ? g.depth : g.q_rows, QT, rag);
    tc_fence_before();
    __syncthreads();
    // The next kernel's blocks start once this grid's blocks hold their tensor memory, and not before: one of them that
    // took the columns first, and then waited for this grid to end, would wait for ever.
    let_next_start();
    if constexpr (CG == 2) cluster_sync();  // its barriers take the other block's arrivals from here on
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_at, 0);  // known to be the same in a warp: see elect_one()

    int tiles = tile_count;
    if (g.ragged == kRowsOfQ) tiles = rag.tiles[g.E] * g.p_tiles;
    const int span = SPLIT ? (int)(gridDim.x) : (int)gridDim.x / CG;  // SPLIT: one tile per cluster
    int split = 1, first_tile = (int)blockIdx.x / CG;
    if constexpr (SPLIT) {
        asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
        first_tile = (int)blockIdx.x / split;
    }
    // Blocks of depth of a tile that this block takes: all, or its share of the groups of four.
    auto depth_of = [&](const Tile& c, int& kb0, int& kb1) {
        kb0 = c.kb0;
        kb1 = c.kb1;
        if constexpr (SPLIT) {
            const int quads = (kb1 - kb0 + 3) / 4;
            const int q0 = (int)((int64_t)quads * (int)rank / split), q1 = (int)((int64_t)quads * ((int)rank + 1) / split);
            kb1 = min(kb1, kb0 + 4 * q1);
            kb0 = kb0 + 4 * q0;
        }
    };

    if (warp == 0) {
        // ---------------------------------------------------------- loads
        int n = 0, s = 0;  // boxes so far, and their place in the ring
        uint32_t parity = 1;  // of the round before: a ring that was never filled is empty
        bool ok = true;
        for (int t = first_tile; ok && t < tiles; t += span) {
            const Tile c = tile_at<PT, QT>(g, rag, t);
            int kb0, kb1;
            depth_of(c, kb0, kb1);
            const int q_rows = CG == 2 ? c.columns / 2 : QT, q_boxes = g.q_mn ? 1 : (q_rows + S::kBox - 1) / S::kBox;
            const int bytes = S::kPBytes + (g.q_mn ? S::kQBytes : q_boxes * S::kBox * 128);
            const int p_row = c.p0 + 128 * (int)pair_rank, q_row = c.q0 + q_rows * (int)pair_rank;
            const int pe = g.p_expert ? c.e : 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = mbar_wait(empty + 8 * s, parity, gave_up);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t at = smem_u32(stages) + s * S::kStageBytes, bar = full + 8 * s;
                    if (leader) mbar_expect_tx(bar, CG * bytes);
                    if (g.p_mn)
                        tma_load<CG == 2>(at, &p_map, bar, p_row, kb * 128, pe);
                    else
                        tma_load<CG == 2>(at, &p_map, bar, kb * 128, p_row, pe);
                    if (g.q_mn)
                        tma_load<CG == 2>(at + S::kPBytes, &q_map, bar, q_row, kb * 128, 0);
                    else
                        for (int i = 0; i < q_boxes; ++i)
                            tma_load<CG == 2>(at + S::kPBytes + i * (S::kBox * 128), &q_map, bar, kb * 128,
                                              q_row + i * S::kBox, 0);
                }
                __syncwarp();
                ++n;
                if (++s == S::kStages) s = 0, parity ^= 1;
            }
        }
        if (!ok && leader) {  // copies in flight land before the block ends
            volatile int again = 0;
            for (int i = n < S::kStages ? 0 : n - S::kStages; i < n; ++i)
                mbar_wait(full + 8 * (i % S::kStages), (i / S::kStages) & 1, &again);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ----------------------------------------------------------- MMAs
        if (leader) {
            int s = 0, it = 0, group = 0;
            uint32_t parity = 0;
            bool ok = true;
            // 32 of depth: 32 bytes along a row, or 32 rows of 128 bytes
            const uint64_t step_p = g.p_mn ? 4096 >> 4 : 32 >> 4, step_q = g.q_mn ? 4096 >> 4 : 32 >> 4;
            const uint64_t desc_p = desc_swizzle128(smem_u32(stages), g.p_mn),
                           desc_q = desc_swizzle128(smem_u32(stages) + S::kPBytes, g.q_mn),
                           desc_s = desc_scales(smem_u32(scales));
            for (int t = first_tile; ok && t < tiles; t += span) {
                const Tile c = tile_at<PT, QT>(g, rag, t);
                int kb0, kb1;
                depth_of(c, kb0, kb1);
                const int depth = __shfl_sync(0xFFFFFFFFu, kb1 - kb0, 0);
                const uint32_t tile_desc = idesc | instruction_columns(__shfl_sync(0xFFFFFFFFu, c.columns, 0));
                const int segment = even_segment(g, depth);
                for (int at = 0; ok && at < depth; at += segment) {
                    const int blocks = min(segment, depth - at);
                    // the accumulator that this tile writes has been taken out
                    if constexpr (QT == 256)
                        ok = it < 1 || mbar_wait(acc_empty, (it - 1) & 1, gave_up);
                    else
                        ok = it < 2 || mbar_wait(acc_empty + 8 * (it & 1), ((it >> 1) - 1) & 1, gave_up);
                    const uint32_t acc = tmem + (it & 1) * S::kAcc1;
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    // Copies the scales of group x of this block's.  That they have arrived says, too, that the
                    // products which used the same bytes and columns before are done.
                    auto scales_of = [&](int x) {
                        const int slot = x % kRing;
                        const bool there = __all_sync(0xFFFFFFFFu, mbar_wait(sc_full + 8 * slot, (x / kRing) & 1, gave_up));
                        tc_fence_after();
                        if (there && elect_one()) {
#pragma unroll
                            for (int h = slot * (kGroup / 4), a = 0; a < (kGroup / 4) * (1 + S::kQAtoms); ++a)
                                copy_scales<CG>(tmem + S::kScaleAt + h * S::kScaleColumns + 4 * a,
                                                desc_s + ((h * S::kScaleBytes + 512 * a) >> 4));
                        }
                        __syncwarp();
                        return there;
                    };
                    ok = ok && scales_of(group);
                    for (int i = 0; ok && i < blocks; ++i) {
                        const uint32_t j = i % kGroup;
                        const uint32_t sfp = tmem + S::kScaleAt + ((group % kRing) * (kGroup / 4) + j / 4) * S::kScaleColumns,
                                       sfq = sfp + 4;
                        ok = ok && mbar_wait(full + 8 * s, parity, gave_up);
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        if (!ok) break;
                        tc_fence_after();
                        const bool last = i + 1 == blocks;
                        if (elect_one()) {
                            const uint64_t dp = desc_p + ((s * S::kStageBytes) >> 4), dq = desc_q + ((s * S::kStageBytes) >> 4);
                            const uint32_t id = tile_desc | scale_byte(j & 3);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_block_scaled<CG>(acc, dp + k * step_p, dq + k * step_q, id, sfp, sfq, i > 0 || k > 0);
                            mma_commit<CG>(empty + 8 * s);
                            if (j == kGroup - 1 || last) mma_commit<CG>(sc_empty + 8 * (group % kRing));
                            if (last) mma_commit<CG>(acc_full + 8 * (it & 1));
                        }
                        __syncwarp();
                        if (++s == S::kStages) s = 0, parity ^= 1;
                        // copied well in front of the products that need them
                        if (j == kGroup - 3 && i + 3 < blocks) ok = scales_of(group + 1);
                        if (j == kGroup - 1) ++group;
                    }
                    if (!ok) break;
                    if (blocks % kGroup) ++group;
                    ++it;
                }
            }
            if (!ok) {  // what has been issued ends before the block does
                volatile int again = 0;
                if (elect_one()) mma_commit<CG>(drained);
                __syncwarp();
                mbar_wait(drained, 0, &again);
            }
        }
        __syncwarp();
    } else if (warp < 4) {
        // --------------------------------------------------------- scales
        auto gather = [&](auto reader, const ScaleSource& src, bool is_p) {
            [[maybe_unused]] const uint32_t arrive_at = CG == 2 ? map_rank(sc_full, 0) : 0;
            int group = 0;
            bool ok = true;
            for (int t = first_tile; ok && t < tiles; t += span) {
                const Tile c = tile_at<PT, QT>(g, rag, t);
                int kb0, kb1;
                depth_of(c, kb0, kb1);
                const int row0 = is_p ? c.p0 + 128 * (int)pair_rank : c.q0;
                if (kb0 < kb1) reader.load(src, c.e, row0, kb0, kb1);
                for (int kb = kb0; kb < kb1; kb += kGroup, ++group) {
                    const int r = group % kRing, round = group / kRing;
                    ok = round == 0 || mbar_wait(sc_empty + 8 * r, (round - 1) & 1, gave_up);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    reader.pack(src, row0, kb, scales + r * (kGroup / 4) * S::kScaleBytes + (is_p ? 0 : 512), S::kScaleBytes);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (CG == 2)
                            mbar_arrive_cluster(arrive_at + 8 * r);
                        else
                            mbar_arrive(sc_full + 8 * r);
                    }
                    if (kb + kGroup < kb1) reader.load(src, c.e, row0, kb + kGroup, kb1);
                }
            }
        };
        if (warp == 2)
            gather(ScaleReader<4>{}, g.sp, true);
        else
            gather(ScaleReader<4 * S::kQAtoms>{}, g.sq, false);
    } else {
        // --------------------------------------------------------- results
        const int band = warp & 3;  // lanes 32 band .. of tensor memory are this warp's
        const uint32_t lanes = (uint32_t)(32 * band) << 16;
        const uint32_t release_at = CG == 2 ? map_rank(acc_empty, 0) : 0;
        constexpr int W = QT < 64 ? QT : 64;  // columns at a time
        int it = 0;
        bool ok = true;
        for (int t = first_tile; t < tiles; t += span) {
            const Tile c = tile_at<PT, QT>(g, rag, t);
            int kb0, kb1;
            depth_of(c, kb0, kb1);
            const bool none = kb0 >= kb1;  // a sum of nothing
            const int segment = even_segment(g, kb1 - kb0);
            for (int seg = kb0; none ? seg == kb0 : seg < kb1; seg += segment) {
                const bool add = seg > kb0;
                const int a = it & 1;
                if (!none) {
                    ok = ok && mbar_wait(acc_full + 8 * a, (it >> 1) & 1, gave_up);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    tc_fence_after();
                    ++it;
                }
                const int row = c.p0 + 128 * (int)pair_rank + 32 * band + lane;  // of P: a column of the output
                const int64_t base = (g.ragged == kDepth ? c.e * g.out_expert : 0) + (ROWS ? row * g.ldo : row);
                const int chunks = QT == 256 ? (c.columns + W - 1) / W : QT / W;
                // eight warps: the even and the odd chunks have four each
                constexpr int kHalves = S::kOutWarps / 4;
                const int half = kHalves == 2 ? (warp - 4) >> 2 : 0;
                bool held = !none;  // the accumulator's shared columns
#pragma unroll 1
                for (int x = half; x < chunks || held; x += kHalves) {
                    // The columns that the two accumulators share come first (the second one's first, the first
                    // one's last): only they hold up the next tile.
                    const int chunk = QT != 256 || a != 0 || chunks != 4 ? x : kHalves == 1 ? (x + 3) & 3 : half == 1 ? x ^ 2 : x;
                    uint32_t v[W];
                    if (!none && ok && x < chunks) {
                        const uint32_t from = tmem + lanes + a * S::kAcc1 + chunk * W;
                        if constexpr (W == 16) {
                            tmem_ld(v, from);
                        } else {
#pragma unroll
                            for (int h = 0; h < W / 32; ++h) tmem_ld(reinterpret_cast<uint32_t(&)[32]>(v[32 * h]), from + 32 * h);
                        }
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int i = 0; i < W; ++i) v[i] = none ? 0u : 0x7FC00000u;
                    }
                    if (held && (QT == 256 || x == chunks - 1)) {
                        held = false;
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            const int bar = QT == 256 ? 0 : a;
                            if constexpr (CG == 2)
                                mbar_arrive_cluster(release_at + 8 * bar);
                            else
                                mbar_arrive(acc_empty + 8 * bar);
                        }
                    }
                    if (x >= chunks) break;
                    if constexpr (SPLIT) {
                        float* part = reinterpret_cast<float*>(stages);  // [QT][128]: every load and MMA is done
#pragma unroll
                        for (int i = 0; i < W; ++i) part[(chunk * W + i) * 128 + 32 * band + lane] = __uint_as_float(v[i]);
                    } else {
                        const int q0 = c.q0 + chunk * W, n = c.q_end - q0;
                        if (add && row < g.p_rows) {  // this thread's own stores of the segments before (fp32)
                            const uint32_t* from = static_cast<const uint32_t*>(g.out) + base + (ROWS ? q0 : q0 * g.ldo);
                            if constexpr (ROWS) {
#pragma unroll
                                for (int h = 0; h < W; h += 32) {
                                    uint32_t old[4][8];  // half of the chunk on its way at once
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        if (h + 8 * k + 8 <= n)
                                            ld32(old[k], from + h + 8 * k);
                                        else
#pragma unroll
                                            for (int i = 0; i < 8; ++i) old[k][i] = h + 8 * k + i < n ? from[h + 8 * k + i] : 0u;
                                    }
#pragma unroll
                                    for (int i = 0; i < 32; ++i) v[h + i] = f32_add(v[h + i], old[i / 8][i % 8]);
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < W; ++i)
                                    if (i < n) v[i] = f32_add(v[i], from[i * g.ldo]);
                            }
                        }
                        uint32_t top = 0;  // NaN results are rare: look for any, then make them canonical
#pragma unroll
                        for (int i = 0; i < W; ++i) top = max(top, v[i] & 0x7FFFFFFFu);
                        if (top > 0x7F800000u)
#pragma unroll
                            for (int i = 0; i < W; ++i) v[i] = canonical(v[i]);
                        if constexpr (ROWS) {
                            // a thread's 64 columns are neighbours: whole sectors of 32 bytes (launch_matmul sees to it that
                            // they are aligned)
                            if (row < g.p_rows) {
                                if (g.out_bf16) {
                                    uint16_t* to = static_cast<uint16_t*>(g.out) + base + q0;
#pragma unroll
                                    for (int h = 0; h < W / 16; ++h) {
                                        uint32_t w[8];
#pragma unroll
                                        for (int i = 0; i < 8; ++i) w[i] = bf16_rne(v[16 * h + 2 * i]) | bf16_rne(v[16 * h + 2 * i + 1]) << 16;
                                        if (16 * h + 16 <= n)
                                            st32(to + 16 * h, w);
                                        else
#pragma unroll
                                            for (int i = 0; i < 16; ++i)
                                                if (16 * h + i < n) to[16 * h + i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
                                    }
                                } else {
                                    uint32_t* to = static_cast<uint32_t*>(g.out) + base + q0;
#pragma unroll
                                    for (int h = 0; h < W / 8; ++h) {
                                        if (8 * h + 8 <= n)
                                            st32(to + 8 * h, reinterpret_cast<uint32_t(&)[8]>(v[8 * h]));
                                        else
#pragma unroll
                                            for (int i = 0; i < 8; ++i)
                                                if (8 * h + i < n) to[8 * h + i] = v[8 * h + i];
                                    }
                                }
                            }
                        } else if (!g.out_bf16) {  // a warp's 32 lanes store 128 neighbouring bytes
                            uint32_t* to = static_cast<uint32_t*>(g.out) + base + q0 * g.ldo;
                            if (row < g.p_rows) {
#pragma unroll
                                for (int i = 0; i < W; ++i, to += g.ldo)
                                    if (i < n) *to = v[i];
                            }
                        } else if (CG == 2) {
                            // Through shared memory, so that a row's 128 features, 256 bytes, are stored together: the
                            // 64 bytes of one warp's lanes make partial lines, and a 256x256 tile took 9.4 us so
                            // (fp32, 128 bytes a warp: 3.1 us; this: 5.3 us).
                            uint16_t* buf = outs + half * (64 * 128);
#pragma unroll
                            for (int i = 0; i < W; ++i) buf[128 * i + 32 * band + lane] = (uint16_t)bf16_rne(v[i]);
                            asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
                            const int part = threadIdx.x & 15, p0 = c.p0 + 128 * (int)pair_rank, left = min(128, g.p_rows - p0);
                            uint16_t* to = static_cast<uint16_t*>(g.out) + base - row + p0 + (int64_t)q0 * g.ldo;
#pragma unroll
                            for (int k = 0; k < W / 8; ++k) {
                                const int i = 8 * k + ((threadIdx.x >> 4) & 7);
                                if (i < n) store_row(to + i * g.ldo, buf + 128 * i, left, part, g.wide);
                            }
                            asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
                        } else {
                            uint16_t* to = static_cast<uint16_t*>(g.out) + base + q0 * g.ldo;
#pragma unroll
                            for (int i = 0; i < W; ++i, to += g.ldo)
                                if (i < n && row < g.p_rows) *to = (uint16_t)bf16_rne(v[i]);
                        }
                    }
                }
            }
        }
        // rows that belong to no expert
        if (g.ragged == kRowsOfQ) {
            const int front = rag.bound[0], behind = rag.bound[g.E];
            for (int64_t i = blockIdx.x; i < (int64_t)front + (g.q_rows - behind); i += gridDim.x) {
                const int64_t row = i < front ? i : behind + (i - front);
                for (int j = threadIdx.x - 128; j < g.p_rows; j += 32 * S::kOutWarps) store_one(g, row * g.ldo + j, 0u);
            }
        }
    }

    if constexpr (SPLIT) {
        // every block adds a share of the columns, in the order of the ranks
        cluster_sync();
        if (first_tile < tiles) {
            const Tile c = tile_at<PT, QT>(g, rag, first_tile);
            const int64_t base = g.ragged == kDepth ? c.e * g.out_expert : 0;
            const uint32_t part = smem_u32(stages);
            const int width = c.q_end - c.q0, j0 = width * (int)rank / split, j1 = width * ((int)rank + 1) / split;
            // four neighbouring rows of P a thread, the sums of all blocks on their way together
            for (int x = threadIdx.x; x < (j1 - j0) * 32; x += S::kThreads) {
                const int j = j0 + (x >> 5), r = (x & 31) * 4;
                float4 v[8];
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    if (s < split) v[s] = ld_cluster_f32x4(map_rank(part + (j * 128 + r) * 4, s));
                float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    if (s < split) sum.x += v[s].x, sum.y += v[s].y, sum.z += v[s].z, sum.w += v[s].w;
                store_four(g, base + (int64_t)(c.q0 + j) * g.ldo + c.p0 + r, g.p_rows - (c.p0 + r), sum);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2 || SPLIT) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_free<CG>(tmem, S::kColumns);
    }
}

// Copies rows of n bytes to rows that begin on 16 bytes, 16 bytes a thread:
// five aligned words of the source, shifted.  What lies behind a row's n bytes
// in the copy is never read (the tensor map ends there).
__global__ void __launch_bounds__(256) repack_kernel(const uint8_t* src, int64_t ld, int64_t rows, int64_t n,
                                                     uint8_t* dst, int64_t ldd) {
    let_next_start();
    wait_for_stream();
    const int64_t pieces = ldd / 16, total = rows * pieces;
    const uint8_t* const end = src + (rows - 1) * ld + n;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < total; u += (int64_t)gridDim.x * 256) {
        int64_t r, c;
        split_index(u, pieces, r, c);
        const uint8_t* from = src + r * ld + 16 * c;
        const uint32_t skip = (uint32_t)(reinterpret_cast<uintptr_t>(from) & 3u);
        uint32_t w[5] = {};
        if (from - skip >= src && from - skip + 20 <= end) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = reinterpret_cast<const uint32_t*>(from - skip)[i];
        } else {  // the matrix's ends, byte by byte into the same places
#pragma unroll
            for (int i = 0; i < 20; ++i) {
                const int at = i - (int)skip;
                if (at >= 0 && at < 16 && 16 * c + at < n) w[i / 4] |= (uint32_t)from[at] << (8 * (i & 3));
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * skip);
        *reinterpret_cast<uint4*>(dst + r * ldd + 16 * c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// ------------------------------------------------------------------- host

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// Boxes of 128 bytes of a row by `box` rows of one operand, of each expert where it is a stack.
bool make_map(CUtensorMap* map, const MatOperand& o, int64_t depth, int64_t E, int box) {
    const int64_t inner = o.mn ? o.rows : depth, outer = o.mn ? depth : o.rows;
    const int64_t experts = o.expert ? E : 1;
    // strides are multiples of 16 bytes; one of a single row, or of a single expert, is not used and may be anything else
    const int64_t ld = outer > 1 || experts > 1 ? o.ld : (inner + 15) / 16 * 16;
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)outer, (cuuint64_t)experts};
    const cuuint64_t strides[2] = {(cuuint64_t)ld, (cuuint64_t)(experts > 1 ? o.expert : ld)};
    const cuuint32_t boxes[3] = {128, (cuuint32_t)box, 1}, steps[3] = {1, 1, 1};
    const EncodeTiled encode = encode_tiled();
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(o.data), dims, strides, boxes,
                            steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

ScaleSource scale_source(const MatOperand& o, int64_t depth) {
    ScaleSource s{};
    s.base = o.scales;
    s.s_row = o.s_row;
    s.s_kb = o.s_kb;
    s.s_expert = o.s_expert;
    s.rows = (int)o.rows;
    s.bytes = o.rows * ceil_div(depth, 128);
    if (o.tiles)
        s.form = kTiles;
    else if (!o.mn)
        s.form = kAlongDepth;
    else
        s.form = o.rows % 4 == 0 && reinterpret_cast<uintptr_t>(o.scales) % 4 == 0 ? kAcrossAligned : kAcrossDepth;
    return s;
}

template <int QT, int CG, bool SPLIT, bool ROWS>
cudaError_t launch(const MatmulArgs& m, int ragged, int columns, int split, cudaStream_t stream) {
    using S = Shape<QT, CG, SPLIT, ROWS>;
    constexpr int PT = 128 * CG;
    const MatOperand &p = ROWS ? m.a : m.b, &q = ROWS ? m.b : m.a;
    Problem g{};
    g.sp = scale_source(p, m.depth);
    g.sq = scale_source(q, m.depth);
    g.offsets = m.offsets;
    g.out = m.out;
    g.ldo = m.ldo;
    g.out_expert = m.out_expert;
    g.E = (int)m.E;
    g.depth = (int)m.depth;
    g.p_rows = (int)p.rows;
    g.q_rows = (int)q.rows;
    g.p_tiles = (int)ceil_div(p.rows, PT);
    g.columns = columns;
    g.segment = SPLIT || m.out_bf16 ? 1 << 26 : kSegment;
    g.q_tiles = (int)ceil_div(q.rows, columns);
    g.ragged = ragged;
    g.p_mn = p.mn;
    g.q_mn = q.mn;
    g.p_expert = p.expert != 0;
    g.out_bf16 = m.out_bf16;
    const int64_t es = m.out_bf16 ? 2 : 4;
    g.wide = reinterpret_cast<uintptr_t>(m.out) % 32 == 0 && m.ldo * es % 32 == 0;
    CUtensorMap pm, qm;
    if (!make_map(&pm, p, m.depth, m.E, 128) || !make_map(&qm, q, m.depth, m.E, q.mn ? 128 : S::kBox))
        return cudaErrorInvalidValue;

    int64_t tiles = (int64_t)g.p_tiles * g.q_tiles * (ragged == kDepth ? m.E : 1);
    if (ragged == kRowsOfQ)  // at most: every expert has a last, partial tile
        tiles = (q.rows / QT + (m.E < q.rows ? m.E : q.rows)) * g.p_tiles;
    if (tiles > INT64_C(0x1FFFFFFF)) return cudaErrorInvalidValue;
    g.whole = (int)tiles;
    if (CG == 2 && ragged == kNone) {
        // a half takes three quarters of a tile's time, and the last round is that much shorter (512x4096x4096 17.0 -> 15.6
        // us, 4099x4096x4096's weight gradient 53.9 -> 51.8, 4099x4096x7184's input gradient 85.2 -> 83.8: means of both sides
        // run in turn, four times for the first and ten for the others)
        const int64_t pairs = sm_count() / 2, rest = tiles % pairs;
        if (rest > 0 && 2 * rest <= pairs) {
            g.whole = (int)(tiles - rest);
            tiles += rest;
        }
    }
    auto kernel = matmul_kernel<QT, CG, SPLIT, ROWS>;
    const size_t smem = S::smem((int)m.E);
    static std::atomic<bool> allowed[kDevices];
    const cudaError_t e = allow_shared_memory(kernel, S::smem(kMostExperts), allowed);
    if (e != cudaSuccess) return e;

    const int64_t room = (int64_t)sm_count() * S::kPerSm / CG;
    const int64_t blocks = SPLIT ? tiles * split : (tiles < room ? tiles : room) * CG;
    const uint32_t idesc = instruction_desc(PT, p.mn, q.mn);
    return launch_overlapped(kernel, dim3((unsigned)blocks), S::kThreads, smem, CG == 2 ? 2 : SPLIT ? split : 0, stream, pm, qm, g,
                             idesc, (int)tiles);
}

}  // namespace

cudaError_t launch_matmul(const MatmulArgs& m, cudaStream_t s) {
    const int ragged = m.grouping == Grouping::DEPTH ? kDepth : m.grouping == Grouping::ROWS ? kRowsOfQ : kNone;
    const int64_t features = m.b.rows, tokens = m.a.rows, blocks = ceil_div(m.depth, 128);
    cudaError_t e;
    // Pairs of blocks and 256x256 tiles where there are rows enough to fill them.  512x4096x4096: 15.2 us, 23.5 in tiles of
    // 128x128 with the depth split; 256: 18.3 and 14.0.  Experts by the rows that each has on average, uneven loads (some
    // have ten times as many as others): 32 of 4096x7184 with 16 rows 150 us in pairs, 170 in single blocks, with 48 169
    // and 212; 32 of 4096x4096 87 and 88, 97 and 101; with 8 rows 124 (4096x7184) and 68 in both, and 64 experts of
    // 2048x2048 48 and 39.  Where every expert has the same number of rows, which a router does not see to, single blocks
    // would stay ahead for longer: 32 of 4096x7184 with 16 rows 163 and 149, with 32 164 and 153, with 50 166 and 170.
    if (tokens > 256 && features > 128 && !(ragged == kRowsOfQ && tokens / m.E < 16)) {
        const int64_t es = m.out_bf16 ? 2 : 4;
        const bool sectors = reinterpret_cast<uintptr_t>(m.out) % 32 == 0 && m.ldo * es % 32 == 0;
        // 8192^3 with the rows as lanes 299 us, as columns 313; 8192x4096x4096 104 and 114 (to fp32 105 and 98); experts'
        // rows are columns for their tiles' width (a 32-expert prompt of 16384 rows: 424 us, 477 as lanes), and so are rows
        // that whole sectors cannot be stored of
        if (ragged != kRowsOfQ && sectors)
            e = launch<256, 2, false, true>(m, ragged, 256, 1, s);
        else
            e = launch<256, 2, false, false>(m, ragged, 256, 1, s);
    } else {
        const int64_t rows = ragged == kRowsOfQ ? ceil_div(tokens, m.E) : tokens;
        // A tile as wide as the rows are many.  Through 8192x8192, 16 rows: 15.8 us in 16 columns, 15.9, 16.1 and 16.9 in 32,
        // 64 and 128; 32 rows: 16.3 in 32, 18.4 in two tiles of 16, 16.6 and 17.4 in 64 and 128; 64 rows: 17.5 in 64, 19.2
        // in two of 32, 18.2 in 128; 128 rows: 20.3 in 128, 21.4 in two of 64.  2048x7168 and 4096x4096 order them alike up
        // to 64 rows, but have 128 in two tiles of 64 in 12.1 and 11.5 us, in one of 128 in 13.0 and 13.6.
        const int qt = m.a.mn || rows > 64 ? 128 : rows > 32 ? 64 : rows > 16 ? 32 : 16;
        const int64_t tiles = ceil_div(features, 128) * ceil_div(tokens, qt), quads = ceil_div(m.depth, 512);
        // as many blocks to a tile's depth as the device has room for at once (two a multiprocessor), and no more than
        // shorten the longest share
        int split = 1;
        if (ragged == kNone)
            for (int x = 2; x <= 8 && x <= quads && tiles * x <= 2 * sm_count(); ++x)
                if (ceil_div(quads, x) < ceil_div(quads, split)) split = x;
        // A share of a cluster is one segment; deeper fp32 results are not split (1x8192x28672: 68.7 us, as bf16, split, 39.6).
        if (!m.out_bf16 && ceil_div(quads, split) * 4 > kSegment) split = 1;
        if (split > 1)
            e = qt == 16   ? launch<16, 1, true, false>(m, ragged, qt, split, s)
                : qt == 32 ? launch<32, 1, true, false>(m, ragged, qt, split, s)
                : qt == 64 ? launch<64, 1, true, false>(m, ragged, qt, split, s)
                           : launch<128, 1, true, false>(m, ragged, qt, split, s);
        else
            e = qt == 16   ? launch<16, 1, false, false>(m, ragged, qt, 1, s)
                : qt == 32 ? launch<32, 1, false, false>(m, ragged, qt, 1, s)
                : qt == 64 ? launch<64, 1, false, false>(m, ragged, qt, 1, s)
                           : launch<128, 1, false, false>(m, ragged, qt, 1, s);
    }
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

cudaError_t launch_repack(const uint8_t* src, int64_t ld, int64_t rows, int64_t n, uint8_t* dst, int64_t ldd,
                          cudaStream_t s) {
    if (rows == 0) return cudaSuccess;
    const int64_t want = ceil_div(rows * (ldd / 16), 256);
    const int64_t most = (int64_t)sm_count() * 32;
    return launch_overlapped(repack_kernel, dim3((unsigned)(want < most ? want : most)), 256, 0, 0, s, src, ld, rows, n, dst,
                             ldd);
}

}  // namespace mxq
