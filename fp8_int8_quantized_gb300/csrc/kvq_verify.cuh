// Attention of a short chunk of new tokens per sequence (drafts under
// verification: 1 to 64 tokens) over the paged quantized cache, the contexts
// split over the whole GPU.
//
// Row r of a (sequence, kv-head): query r / G of the chunk, q-head r % G of the
// kv-head's group.  With P = ctx - n committed tokens,
//   z_rt = sm_scale * q_r . k_t,   a_rt = 1 for t < P, else bit t - P of the
//   query's mask (causal when there is none),
//   o_r = sum_t a_rt e^(z_rt - m_r) v_t / sum_t a_rt e^(z_rt - m_r)
// in one pass over the cache with a running maximum and sum; a row that sees
// nothing gives zeros.  The FP8 scale and the INT8 / INT4 row or group scales
// are taken out of the products: logits take s_K, weights (INT8 / INT4) or
// outputs (FP8) take s_V.  Products are fp16 x fp16, sums fp32, and the weights
// enter P V as an fp16 pair (value + residual, 22 bits of the larger ones: kUp, log2_scale).
//
// What bounds it: every cached byte is read once (2 D bytes per token and
// kv-head for 8-bit codes) against 4 D flops per row and token: the stream from
// HBM should, but the conversion of the codes to fp16 and the softmax take
// nearly as long as the bytes.  These kernels use mma.sync; they serve head_dim 64 and
// batches above kMaxTcBatch, and kvq_verify_tc.cuh the rest.  head_dim 128 with
// E4M3 codes, 32 sequences of 8192 tokens, 8 kv-heads: 1 row 127 us (4.2 TB/s),
// 32 rows 225 us; INT8 with 16 x 4096 tokens, 40 kv-heads, 8 rows: 160 us (L2
// flushed before each call).  head_dim 64, 32 x 8192 tokens, 8 kv-heads, calls back to
// back: E4M3 1 row 88 us (3.1 TB/s), 32 rows 127; INT8 8 rows 103, 32 rows 150, with
// 16-channel groups 212; INT4 32 rows 147, with 16-channel groups 263.
//
// Work.  A row tile is RT (8, 16 or 32) rows of one (sequence, kv-head); the
// tiles of 32 tokens of all row tiles, in (row tile, sequence, kv-head, token)
// order, form flat lists, one per row-tile number.  Every list gets CTAs in
// proportion to its length, and cuts its tiles into equal contiguous ranges,
// one per team.  A team is one warp, or all warps of a CTA when a range would
// be only a few tiles long (the partial results of 32 rows are as large as two
// tiles): its warps take the range's tiles in turn and merge their sums in
// shared memory.  (Row tiles 0 and 1 of a sequence walk the same cache rows in
// step on different SMs, so the second one finds them in L2.)
//
// A team walks segments: the part of its range in one (row tile, sequence,
// kv-head).  A segment that holds all tiles of it is written straight to the
// output; else its (m, sum, accumulator) goes to one of the team's two partial
// slots (0: it starts inside, 1: it starts at the first tile), and the team of
// the first part leaves a header for verify_reduce_kernel.  So at most two
// partials per team exist, whatever the context length.
//
// Per warp: a ring of kStages tiles (two 16-row TMA boxes of K and of V each,
// swizzled so that ldmatrix is free of bank conflicts, and the row scales by
// bulk copies), refilled right after use across segment borders.  Q K^T is
// computed with the rows as M (16) and tokens as N (8), so its accumulator is
// already the B operand of out^T = V^T P^T (channels as M, rows as N).  The
// channel order inside a 16-byte chunk is permuted the same way for Q and K, so
// one register of codes is one fragment.  The rows' Q fragments lie in shared
// memory in the order the lanes load them.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "kvq_device.cuh"
#include "kvq_spec.h"

namespace kvq {
namespace verify {

constexpr int kTile = 32;     // tokens per stage
constexpr int kBox = 16;      // rows per TMA box
constexpr int kStages = 2;    // per warp
constexpr int kMaxClasses = 64;   // row tiles per (sequence, kv-head): 64 queries x 8 heads / 8 rows
constexpr float kLog2e = 1.4426950408889634f;
// A row's running maximum moves only when a tile exceeds it by more than 2^8,
// so weights stay below 2^8 and hardly a tile rescales anything.
constexpr float kLazy = 8.0f;
// Weights are stored times 2^kUp, a row's largest in 2^6 .. 2^14: an fp16 pair holds 22 bits of a
// weight from 2^-3 on, below that an absolute 2^-25, 2^-31 of the largest.  (Where one token of small V
// takes most of the softmax, 8000 tokens, INT4 with 64-channel groups: 2.7e-3 of the result with
// weights times 2^-6, 2.1e-4 with 2^6, which is the rounding of the output.)
constexpr float kUp = 6.0f;
// Where a weight carries its token's V scale, "largest" is that of the product: the running maximum is
// of z + log2 |s_V| (the largest of the row's groups), so that the pair's range does not depend on how
// large V is.  The sum of the weights without the scale is held in fp32 and takes the same factors.  (With
// the maximum of z alone and fixed factors 2^-2 and 2^-6, INT8 and INT4, 8000 tokens: 2.4e-3 of
// the result for V of 2^-7, 2e-2 for 2^-10; now 2.2e-4 and 9e-4, the rounding of the output.)
// Bounded by 2^-40 (all values below fp16's smallest) and 2^40, NaN too: rows of zeros have scale 0.
__device__ __forceinline__ float log2_scale(float s) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fabsf(s)));
    return fminf(fmaxf(r, -40.f), 40.f);
}

__device__ __forceinline__ float warp_max(float x) {   // over the warp; NaN does not count
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}
__device__ __forceinline__ float ldsf(uint32_t a) {
    float r;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(a));
    return r;
}
// Four 8x8 matrices of 16-bit elements, row addresses from lanes 8m .. 8m + 7.
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ uint32_t hfma2_const(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// Four 8-bit codes -> fp16 pairs of bytes (0, 1) and (2, 3), exact.
template <int FMT>
__device__ __forceinline__ void dec4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (FMT == INT8) {
        const uint32_t x = w ^ 0x80808080u;   // code + 128
        lo = hsub2_exact(prmt(x, 0x64646464u, 0x4140u), 0x64806480u);   // 1024 + 128 + code - 1152
        hi = hsub2_exact(prmt(x, 0x64646464u, 0x4342u), 0x64806480u);
    } else if constexpr (FMT == E5M2) {   // an fp16's upper byte (the conversion runs at a quarter of prmt's rate)
        lo = prmt(w, 0u, 0x1404u);
        hi = prmt(w, 0u, 0x3424u);
    } else {
        dec_fp8x4<FMT>(w, lo, hi);
    }
}
// INT4: the low (high) nibbles of bytes 0 and 2 of w ^ 0x88.. (code + 8) -> fp16 pair, exact.
__device__ __forceinline__ uint32_t nib_lo(uint32_t x) { return hsub2_exact((x & 0x000F000Fu) | 0x64006400u, 0x64086408u); }
__device__ __forceinline__ uint32_t nib_hi(uint32_t x) {   // 1024 + 16 n -> n - 8
    return hfma2_const((x & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u);
}

// fp16 pair of two weights, and the fp16 pair of what it leaves out.
__device__ __forceinline__ void split2(float p0, float p1, uint32_t& hi, uint32_t& lo) {
    hi = pack_f16x2(p0, p1);
    const float2 h = f16x2_to_f32x2(hi);
    lo = pack_f16x2(p0 - h.x, p1 - h.y);
}

// Position in a class's flat tile list.
struct Walk {
    int b, kvh, t, n;   // n: tiles of the sequence
};

// One sequence of the call: n new queries from row q0 on, ctx cached tokens;
// tiles 0 when it has nothing to do or its lengths are not usable.
struct Seq {
    int q0, n, ctx, tiles;
};

template <int TT = kTile>
__device__ __forceinline__ Seq seq_of(const VerifyArgs& a, int b, bool record) {
    Seq s;
    s.q0 = __ldg(a.query_start + b);
    s.n = __ldg(a.query_start + b + 1) - s.q0;
    s.ctx = __ldg(a.context_lens + b);
    s.tiles = 0;
    if (s.n == 0) return s;
    const int64_t cap = min((int64_t)a.max_context_len, (int64_t)a.max_blocks_per_seq * a.cache.block_size);
    if (s.n < 0 || s.n > a.max_query_len || s.q0 < 0 || (int64_t)s.q0 + s.n > a.num_q_tokens || s.n > s.ctx || s.ctx > cap) {
        if (record) record_error(a.err, DEV_ERR_RANGE, b);
        s.n = 0;
        return s;
    }
    s.tiles = (int)(((unsigned)s.ctx + TT - 1) / TT);
    return s;
}

__device__ __forceinline__ Walk locate(const int* S, int B, int Hkv, int f) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (Hkv * S[mid] <= f) lo = mid; else hi = mid - 1;
    }
    Walk w;
    w.b = lo;
    w.n = S[lo + 1] - S[lo];
    const int r = f - Hkv * S[lo];
    w.kvh = r / w.n;
    w.t = r - w.kvh * w.n;
    return w;
}

// This CTA's class (row-tile number), its place among the class's CTAs, and
// the scan of the class's tiles: S[b] = tiles of sequences 0 .. b - 1 that have
// more than cls row tiles.  Called by all threads of the CTA.
struct ClassOf {
    int cls, cta, ctas;   // cls -1: nothing to do
};

template <int THREADS, int TT>
__device__ __forceinline__ ClassOf scan_class(const VerifyArgs& a, int row_tiles, int RT, int* S) {
    __shared__ int hist[kMaxClasses + 1], wsum[THREADS / 32], place[3];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int B = a.batch, G = a.num_q_heads / a.cache.num_kv_heads;
    for (int i = threadIdx.x; i <= kMaxClasses; i += THREADS) hist[i] = 0;
    __syncthreads();
    const int per = (B + THREADS - 1) / THREADS;
    const int b0 = min(B, (int)threadIdx.x * per), b1 = min(B, b0 + per);
    for (int b = b0; b < b1; ++b) {
        const Seq s = seq_of<TT>(a, b, blockIdx.x == 0);
        if (s.tiles) atomicAdd(&hist[(s.n * G + RT - 1) / RT], s.tiles);   // whole numbers: any order
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        // tiles of class k: those of sequences with more than k row tiles
        int64_t total = 0;
        int run = 0, classes = 0;
        for (int k = row_tiles; k >= 1; --k) {
            run += hist[k];
            hist[k] = run;   // now the tiles of class k - 1
            total += run;
            classes += run > 0;
        }
        // one CTA per class with work, the others in proportion to the tiles
        int base = 0;
        place[0] = -1;
        place[1] = place[2] = 0;
        for (int k = 0; k < row_tiles && hist[k + 1] > 0; ++k) {
            const int m = 1 + (int)((int64_t)((int)gridDim.x - classes) * hist[k + 1] / total);
            if ((int)blockIdx.x >= base && (int)blockIdx.x < base + m) {
                place[0] = k;
                place[1] = (int)blockIdx.x - base;
                place[2] = m;
            }
            base += m;
        }
    }
    __syncthreads();
    const ClassOf c{place[0], place[1], place[2]};
    int local = 0;
    for (int b = b0; b < b1; ++b) {
        const Seq s = seq_of<TT>(a, b, false);
        local += s.n * G > c.cls * RT ? s.tiles : 0;
    }
    int x = local;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    int run = x - local;
    for (int w = 0; w < warp; ++w) run += wsum[w];
    for (int b = b0; b < b1; ++b) {
        const Seq s = seq_of<TT>(a, b, false);
        S[b] = run;
        run += s.n * G > c.cls * RT ? s.tiles : 0;
    }
    if (threadIdx.x == THREADS - 1) S[B] = run;
    __syncthreads();
    return c;
}

template <int FMT, int D, int RT>
struct Shape {
    static constexpr bool I4 = FMT == INT4, kScaled = FMT == INT8 || FMT == INT4;
    static constexpr int RB = row_bytes(FMT, D), CH = RB / 16;   // bytes, 16-byte chunks per row
    static constexpr int KS = D / 16, MT = D / 16;               // k-steps of Q K^T, m-tiles of P V
    static constexpr int NQ = (RT + 15) / 16, NT = RT / 8;       // m-tiles of Q K^T, n-tiles of P V
    static constexpr int kWarps = 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kTileBytes = kTile * RB;
    static constexpr int kQBytes = KS * NQ * 32 * (RT == 8 ? 8 : 16);   // a team's Q fragments
    // merge buffer of a whole-CTA team: [warp][RT][32 channels], rows padded to 36 floats
    static constexpr int kMergeRow = 36;
    static constexpr int kMergeBytes = kWarps * RT * kMergeRow * 4;
    static constexpr int kMl = kQBytes + kMergeBytes, kOneTeam = kMl + kWarps * RT * 8;   // then (m, sum) per warp and row
    static constexpr int kTeamBytes = kWarps * kQBytes > kOneTeam ? kWarps * kQBytes : kOneTeam;
};

// Shared memory of one CTA, from a 1024-byte aligned base: tile rings, scale
// rings, Q fragments (one set per warp; or one set, the merge buffer and the
// warps' (m, sum) of a whole-CTA team), barriers, the scan of tiles.
struct Layout {
    int scales, team, full, scan, total;
    __host__ __device__ Layout(int warps, int tile_bytes, int team_bytes, bool scaled, int ng, int B) {
        scales = warps * kStages * 2 * tile_bytes;
        team = scales + (scaled ? warps * kStages * 2 * kTile * 4 * ng : 0);
        full = team + team_bytes;
        scan = full + warps * kStages * 8;
        total = scan + (B + 1) * 4;
    }
};

// NG: 1 (a scale per row or tensor) or 4 (two or four group scales per row).
template <int FMT, int D, int RT, int NG>
__global__ void __launch_bounds__(Shape<FMT, D, RT>::kThreads, 1)
    verify_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const VerifyArgs a,
                  const VerifyPlan plan) {
    using X = Shape<FMT, D, RT>;
    constexpr int W = X::kWarps, RB = X::RB, CH = X::CH, NQ = X::NQ, NT = X::NT, MT = X::MT;
    constexpr bool I4 = X::I4, kScaled = X::kScaled;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int B = a.batch, Hkv = a.cache.num_kv_heads, BS = a.cache.block_size, G = a.num_q_heads / Hkv;
    const int ng = a.cache.ngroups;
    const Layout L(W, X::kTileBytes, X::kTeamBytes, kScaled, ng, B);
    const bool solo = plan.team == 1;   // every warp is a team of its own
    const int team = solo ? blockIdx.x * W + warp : blockIdx.x;
    int4* hdr = reinterpret_cast<int4*>(a.ws) + team;   // {sequence, kv-head, row tile, later parts}
    float2* ws_ml = reinterpret_cast<float2*>(a.ws + verify_ml_off(plan.teams));
    float* ws_acc = reinterpret_cast<float*>(a.ws + verify_acc_off(plan.teams, RT));
    int* S = reinterpret_cast<int*>(smem + L.scan);
    griddep_wait();
    griddep_launch();

    if (threadIdx.x < W * kStages) mbar_init(reinterpret_cast<uint64_t*>(smem + L.full) + threadIdx.x, 1);
    fence_barrier_init();
    const ClassOf co = scan_class<X::kThreads, kTile>(a, plan.row_tiles, RT, S);
    const int cls = co.cls, cta_s = co.cta, ctas_s = co.ctas;
    // ---- this team's range of the class's list -------------------------------
    const int T = cls < 0 ? 0 : Hkv * S[B];
    const int nteams = solo ? ctas_s * W : ctas_s;
    const int ct = solo ? cta_s * W + warp : cta_s;   // team within the class
    const int len = T > 0 ? T / nteams : 0, extra = T > 0 ? T % nteams : 0;
    const int lo = T > 0 ? ct * len + min(ct, extra) : 0;
    const int hi = T > 0 ? lo + len + (ct < extra ? 1 : 0) : 0;
    const int step = solo ? 1 : W, wi = solo ? 0 : warp;   // this warp takes tiles lo + wi, + step, ...
    const bool lead = solo ? lane == 0 : threadIdx.x == 0;
    if (lo >= hi) {   // whole teams only: no barrier of a team is skipped
        if (lead) *hdr = make_int4(0, 0, 0, 0);
        return;
    }
    auto team_sync = [&]() { if (solo) __syncwarp(); else __syncthreads(); };

    const uint32_t tiles_u32 = smem_u32(smem) + warp * kStages * 2 * X::kTileBytes;
    const uint32_t sc_stage = 2 * kTile * 4 * ng;   // bytes of a stage's K and V scales
    const uint32_t scales_u32 = smem_u32(smem) + L.scales + warp * kStages * sc_stage;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L.full) + warp * kStages;
    uint8_t* qfrag = smem + L.team + (solo ? warp * X::kQBytes : 0);
    const uint32_t qf_u32 = smem_u32(qfrag);
    float* merge = reinterpret_cast<float*>(smem + L.team + X::kQBytes);
    float2* ml_s = reinterpret_cast<float2*>(smem + L.team + X::kMl);
    const uint64_t pol = policy_evict_first();
    // several row tiles read the same rows: leave them in L2 for the others
    const bool keep = plan.row_tiles > 1;

    // ---- issue side: tile k of this warp is flat tile lo + wi + k * step -----
    const int cnt = (hi - lo - wi + step - 1) / step > 0 ? (hi - lo - wi + step - 1) / step : 0;   // this warp's tiles
    // block ids of the boxes of tiles [k0, k0 + 16): lane j holds box j % 2 of tile k0 + j / 2
    auto load_id = [&](int k0) -> int {
        const int k = k0 + (lane >> 1);
        if (k >= cnt) return 0;
        const Walk w = locate(S, B, Hkv, lo + wi + k * step);
        const int tok = w.t * kTile + (lane & 1) * kBox;
        if (tok >= __ldg(a.context_lens + w.b)) return 0;
        return __ldg(a.block_tables + (int64_t)w.b * a.max_blocks_per_seq + tok / BS);
    };
    int idc = load_id(0), idn = load_id(16);
    if (lane == 0) {
        prefetch_tmap(&tmk);
        prefetch_tmap(&tmv);
    }
    const bool big_box = BS >= kTile;
    const uint32_t box_tx = 2 * kBox * RB + (kScaled ? 2 * kBox * 4 * ng : 0);
    Walk iw = cnt > 0 ? locate(S, B, Hkv, lo + wi) : Walk{0, 0, 0, 1};
    int ik = 0, ist = 0;   // next tile to issue, its stage
    int ck = 0, cst = 0;   // next tile to consume, its stage
    uint32_t cph = 0;
    auto issue_ready = [&]() {
        while (ik < cnt && ik - ck < kStages) {
            const int id0 = __shfl_sync(0xFFFFFFFFu, idc, (2 * ik) & 31), id1 = __shfl_sync(0xFFFFFFFFu, idc, (2 * ik + 1) & 31);
            const int tok0 = iw.t * kTile;
            const int nbox = big_box ? 2 : (__ldg(a.context_lens + iw.b) - tok0 > kBox ? 2 : 1);
            uint64_t* fb = &full[ist];
            if (lane == 0) mbar_arrive_expect_tx(fb, nbox * box_tx);
            // lanes 0-3: boxes of K and V; 4-7: their scales (one 32-row copy each when a block holds the tile)
            const int bx = lane & 1, which = (lane >> 1) & 1;
            if (lane < (kScaled ? 8 : 4) && bx < (big_box ? 1 : nbox)) {
                int blk = bx ? id1 : id0;
                if (blk < 0 || blk >= a.cache.num_blocks) {
                    record_error(a.err, DEV_ERR_RANGE, blk);
                    blk = 0;   // the pipeline goes on with a block that exists
                }
                const int row = (blk * Hkv + iw.kvh) * BS + ((tok0 + bx * kBox) & (BS - 1));
                if (lane < 4) {
                    const uint32_t dst = tiles_u32 + ist * (2 * X::kTileBytes) + which * X::kTileBytes + bx * kBox * RB;
                    if (keep) {
                        asm volatile(
                            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(which ? &tmv : &tmk), "r"(0), "r"(row),
                            "r"(smem_u32(fb))
                            : "memory");
                    } else {
                        tma_load_2d_u32(dst, which ? &tmv : &tmk, 0, row, fb, pol);
                    }
                } else {
                    const uint32_t sb = (big_box ? kTile : kBox) * 4 * ng;
                    const uint32_t dst = scales_u32 + ist * sc_stage + which * (kTile * 4 * ng) + bx * (kBox * 4 * ng);
                    bulk_load_u32(dst, (which ? a.cache.v_scales : a.cache.k_scales) + (int64_t)row * ng, sb, fb, pol);
                }
            }
            ++ik;
            ist = ist + 1 == kStages ? 0 : ist + 1;
            if (ik < cnt) {
                iw.t += step;
                while (iw.t >= iw.n) {   // past the end of the pair: the next one with tiles
                    iw.t -= iw.n;
                    if (++iw.kvh == Hkv) {
                        iw.kvh = 0;
                        do { ++iw.b; } while (iw.b < B && S[iw.b + 1] == S[iw.b]);
                        iw.n = iw.b < B ? S[iw.b + 1] - S[iw.b] : 0x7FFFFFFF;
                    }
                }
            }
            if ((ik & 15) == 0) {
                idc = idn;
                idn = load_id(ik + 16);
            }
        }
    };
    issue_ready();

    const float s_fp8 = (!kScaled && a.scale) ? __ldg(a.scale) : 1.0f;
    const float qk_scale = a.sm_scale * s_fp8 * kLog2e;   // logits in log2 units
    constexpr int SUB = (I4 && D == 64 && NG == 4) ? 2 : 1;   // scale groups inside a 16-byte chunk
    constexpr int CPG = NG == 1 ? CH : (CH >= NG ? CH / NG : 1);   // chunks per scale group
    // byte offset of this lane's row in chunk ch of a 32-row tile (rows = tokens)
    auto chunk_off = [&](int ch) -> uint32_t {
        const int sw = RB == 128 ? (lane & 7) : RB == 64 ? ((lane >> 1) & 3) : ((lane >> 2) & 1);
        return lane * RB + ((ch ^ sw) << 4);
    };

    float acc[NT][MT][4];
    float m[NT], l[NT];   // rows 8 n + g
    bool failed = false;

    int f = lo;
    Walk sw = locate(S, B, Hkv, lo);
    while (f < hi) {
        // ---------------------------------------------------- segment start ----
        const Seq sq = seq_of(a, sw.b, false);
        const int P = sq.ctx - sq.n, R = min(RT, sq.n * G - cls * RT);   // live rows of the tile
        const int seg = min(hi - f, sw.n - sw.t);                         // tiles of the segment
        const unsigned long long live = sq.n >= 64 ? ~0ull : (1ull << sq.n) - 1ull;
        // global row of tile row r: (query, head)
        auto out_row = [&](int r) -> int64_t {
            const int rr = cls * RT + r;
            return (int64_t)(sq.q0 + rr / G) * a.num_q_heads + sw.kvh * G + rr % G;
        };
        {   // Q fragments: lane (g, c) of m-tile qt, k-step ks holds rows 16 qt + g and + 8
            const int tid = solo ? lane : threadIdx.x, nthr = solo ? 32 : X::kThreads;
            constexpr int kPieces = X::KS * NQ * 32;
            for (int i = tid; i < (I4 ? kPieces / 2 : kPieces); i += nthr) {
                const int ln = i & 31, qt = (i >> 5) % NQ, ks = (i >> 5) / NQ, qg = ln >> 2, qc = ln & 3;
                const int ra = 16 * qt + qg, rb = ra + 8;
                if constexpr (I4) {   // 8 channels of chunk ks: k-steps 2 ks and 2 ks + 1
                    uint4 x = make_uint4(0, 0, 0, 0), y = x;
                    if (ra < R) x = *reinterpret_cast<const uint4*>(a.q + out_row(ra) * D + 32 * ks + 8 * qc);
                    if (rb < R) y = *reinterpret_cast<const uint4*>(a.q + out_row(rb) * D + 32 * ks + 8 * qc);
                    // channel pairs (0, 4), (1, 5) | (2, 6), (3, 7)
                    const uint32_t x04 = prmt(x.x, x.z, 0x5410u), x15 = prmt(x.x, x.z, 0x7632u);
                    const uint32_t x26 = prmt(x.y, x.w, 0x5410u), x37 = prmt(x.y, x.w, 0x7632u);
                    const uint32_t y04 = prmt(y.x, y.z, 0x5410u), y15 = prmt(y.x, y.z, 0x7632u);
                    const uint32_t y26 = prmt(y.y, y.w, 0x5410u), y37 = prmt(y.y, y.w, 0x7632u);
                    const int s0 = (2 * ks * NQ + qt) * 32 + ln, s1 = ((2 * ks + 1) * NQ + qt) * 32 + ln;
                    if constexpr (RT == 8) {
                        reinterpret_cast<uint2*>(qfrag)[s0] = make_uint2(x04, x15);
                        reinterpret_cast<uint2*>(qfrag)[s1] = make_uint2(x26, x37);
                    } else {
                        reinterpret_cast<uint4*>(qfrag)[s0] = make_uint4(x04, y04, x15, y15);
                        reinterpret_cast<uint4*>(qfrag)[s1] = make_uint4(x26, y26, x37, y37);
                    }
                } else {              // channels 16 ks + 4c .. + 3
                    uint2 x = make_uint2(0, 0), y = x;
                    if (ra < R) x = *reinterpret_cast<const uint2*>(a.q + out_row(ra) * D + 16 * ks + 4 * qc);
                    if (rb < R) y = *reinterpret_cast<const uint2*>(a.q + out_row(rb) * D + 16 * ks + 4 * qc);
                    if constexpr (RT == 8) reinterpret_cast<uint2*>(qfrag)[i] = x;
                    else reinterpret_cast<uint4*>(qfrag)[i] = make_uint4(x.x, y.x, x.y, y.y);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n] = -INFINITY;
            l[n] = 0.f;
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[n][i][0] = acc[n][i][1] = acc[n][i][2] = acc[n][i][3] = 0.f;
        }
        team_sync();

        // ------------------------------------------------------ its tiles ----
        while (ck < cnt && lo + wi + ck * step < f + seg) {
            const int t0 = (sw.t + (lo + wi + ck * step - f)) * kTile;   // first token of the tile
            if (!failed && !mbar_wait(&full[cst], cph, nullptr)) {
                if (lane == 0) record_error(a.err, DEV_ERR_TIMEOUT, lo + wi + ck * step);
                failed = true;   // no more loads or products; the team's barriers are still met
                int st = cst;
                uint32_t ph = cph;
                for (int k = ck; k < ik; ++k) {   // let the copies in flight land
                    mbar_wait(&full[st], ph, nullptr);
                    st = st + 1 == kStages ? 0 : st + 1;
                    ph ^= st == 0 ? 1u : 0u;
                }
            }
            if (!failed) {
                const uint32_t kt = tiles_u32 + cst * (2 * X::kTileBytes), vt = kt + X::kTileBytes;
                const uint32_t sk = scales_u32 + cst * sc_stage, sv = sk + kTile * 4 * ng;
                const bool masked = t0 + kTile > P;
                // ---- logits: s[qt][j][2h + e] = row 16 qt + 8 h + g, token 8 j + 2c + e
                float s[NQ][4][4];
#pragma unroll
                for (int qt = 0; qt < NQ; ++qt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[qt][j][0] = s[qt][j][1] = s[qt][j][2] = s[qt][j][3] = 0.f;
                auto qk = [&](float (&d)[NQ][4][4], int ks, int j, uint32_t k0, uint32_t k1, const uint4 (&qa)[NQ]) {
#pragma unroll
                    for (int qt = 0; qt < NQ; ++qt)
                        mma_16816(d[qt][j], qa[qt].x, qa[qt].y, qa[qt].z, qa[qt].w, k0, k1);
                };
                auto load_q = [&](int ks, uint4 (&qa)[NQ]) {
#pragma unroll
                    for (int qt = 0; qt < NQ; ++qt) {
                        if constexpr (RT == 8) {
                            const uint2 x = lds64(qf_u32 + (ks * 32 + lane) * 8);
                            qa[qt] = make_uint4(x.x, 0u, x.y, 0u);
                        } else {
                            qa[qt] = lds128(qf_u32 + ((ks * NQ + qt) * 32 + lane) * 16);
                        }
                    }
                };
                auto qk_chunk = [&](float (&d)[NQ][4][4], int ch, int sub) {
                    uint32_t r[4];
                    ldsm4(kt + chunk_off(ch), r);
#pragma unroll
                    for (int hk = 0; hk < (I4 ? 2 : 1); ++hk) {
                        uint4 qa[NQ];
                        load_q((I4 ? 2 * ch : ch) + hk, qa);
                        if constexpr (SUB == 2) {   // only the channels of the sub-group: lanes 2 sub, 2 sub + 1
                            if ((c >> 1) != sub) {
#pragma unroll
                                for (int qt = 0; qt < NQ; ++qt) qa[qt] = make_uint4(0, 0, 0, 0);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t k0, k1;
                            if constexpr (I4) {
                                const uint32_t x = hk ? (r[j] ^ 0x88888888u) >> 8 : r[j] ^ 0x88888888u;
                                k0 = nib_lo(x);
                                k1 = nib_hi(x);
                            } else {
                                dec4<FMT>(r[j], k0, k1);
                            }
                            qk(d, 0, j, k0, k1, qa);
                        }
                    }
                };
                if constexpr (NG == 1) {
#pragma unroll
                    for (int ch = 0; ch < CH; ++ch) qk_chunk(s, ch, 0);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float k0 = qk_scale, k1 = qk_scale;
                        if (kScaled) {
                            k0 *= ldsf(sk + 4 * (8 * j + 2 * c));
                            k1 *= ldsf(sk + 4 * (8 * j + 2 * c) + 4);
                        }
#pragma unroll
                        for (int qt = 0; qt < NQ; ++qt) {
                            s[qt][j][0] *= k0; s[qt][j][1] *= k1; s[qt][j][2] *= k0; s[qt][j][3] *= k1;
                        }
                    }
                } else {
#pragma unroll
                    for (int gi = 0; gi < NG; ++gi) {
                        float d[NQ][4][4];
#pragma unroll
                        for (int qt = 0; qt < NQ; ++qt)
#pragma unroll
                            for (int j = 0; j < 4; ++j) d[qt][j][0] = d[qt][j][1] = d[qt][j][2] = d[qt][j][3] = 0.f;
                        if constexpr (SUB == 2) {
                            qk_chunk(d, gi >> 1, gi & 1);
                        } else {
#pragma unroll
                            for (int x = 0; x < CPG; ++x) qk_chunk(d, gi * CPG + x, 0);
                        }
                        const int gs = (gi * ng) >> 2;   // the stored scale of this quarter of the row
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t at = sk + 4 * ((8 * j + 2 * c) * ng + gs);
                            const float k0 = qk_scale * ldsf(at), k1 = qk_scale * ldsf(at + 4 * ng);
#pragma unroll
                            for (int qt = 0; qt < NQ; ++qt) {
                                s[qt][j][0] = fmaf(d[qt][j][0], k0, s[qt][j][0]);
                                s[qt][j][1] = fmaf(d[qt][j][1], k1, s[qt][j][1]);
                                s[qt][j][2] = fmaf(d[qt][j][2], k0, s[qt][j][2]);
                                s[qt][j][3] = fmaf(d[qt][j][3], k1, s[qt][j][3]);
                            }
                        }
                    }
                }
                // ---- mask: bit u of word[n] = row 8 n + g sees token t0 + u
                uint32_t word[NT];
                if (masked) {
                    const int base = t0 - P;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int qi = (cls * RT + 8 * n + g) / G;
                        unsigned long long bits = 0;
                        if (8 * n + g < R)
                            bits = (a.tree_mask ? __ldg(a.tree_mask + sq.q0 + qi) : (qi >= 63 ? ~0ull : (2ull << qi) - 1ull)) & live;
                        word[n] = base >= 0 ? (base < 64 ? (uint32_t)(bits >> base) : 0u)
                                            : (uint32_t)(bits << -base) | ((1u << -base) - 1u);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (!((word[n] >> (8 * j + 2 * c + e)) & 1u)) s[n >> 1][j][2 * (n & 1) + e] = -INFINITY;
                    }
                }
                // ---- running maximum (of the weights with V's scale), weights, sums
                float mx[NT];
                bool raise = false;
                [[maybe_unused]] float lv = 0.f, lv_top = 0.f;   // log2 of the scale of the lane's token; the tile's largest
                if constexpr (kScaled) {
                    if (NG == 1) {
                        lv = ldsf(sv + 4 * lane);
                    } else if (ng == 4) {
                        const uint4 x = lds128(sv + 16 * lane);
                        lv = fmaxf(fmaxf(fabsf(__uint_as_float(x.x)), fabsf(__uint_as_float(x.y))),
                                   fmaxf(fabsf(__uint_as_float(x.z)), fabsf(__uint_as_float(x.w))));
                    } else {
                        const uint2 x = lds64(sv + 8 * lane);
                        lv = fmaxf(fabsf(__uint_as_float(x.x)), fabsf(__uint_as_float(x.y)));
                    }
                    lv = log2_scale(lv);
                    lv_top = warp_max(lv);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mx[n] = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 4; ++j) mx[n] = fmaxf(mx[n], fmaxf(s[n >> 1][j][2 * (n & 1)], s[n >> 1][j][2 * (n & 1) + 1]));
                    if (kScaled) {
                        raise |= mx[n] + lv_top > m[n] + kLazy;
                    } else {
                        mx[n] = fmaxf(mx[n], __shfl_xor_sync(0xFFFFFFFFu, mx[n], 1));
                        mx[n] = fmaxf(mx[n], __shfl_xor_sync(0xFFFFFFFFu, mx[n], 2));
                    }
                }
                if constexpr (kScaled) {
                    // Most tiles stay below by the largest logit and the largest scale together; the others' maxima are of
                    // the sums token by token (so in every tile: INT8, 32 x 8192 tokens, head_dim 64, 8 heads, 8 rows,
                    // 102.8 -> 104.6 us; 16-channel groups, 32 rows, 212 -> 219).
                    const bool some = __any_sync(0xFFFFFFFFu, raise);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mx[n] = -INFINITY;
                    if (some) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float x = __shfl_sync(0xFFFFFFFFu, lv, 8 * j + 2 * c + e);
#pragma unroll
                                for (int n = 0; n < NT; ++n) mx[n] = fmaxf(mx[n], s[n >> 1][j][2 * (n & 1) + e] + x);
                            }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mx[n] = fmaxf(mx[n], __shfl_xor_sync(0xFFFFFFFFu, mx[n], 1));
                            mx[n] = fmaxf(mx[n], __shfl_xor_sync(0xFFFFFFFFu, mx[n], 2));
                        }
                    }
                }
                float alpha[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    alpha[n] = 1.f;
                    if (mx[n] > m[n] + kLazy) {
                        alpha[n] = fast_exp2(m[n] - mx[n]);
                        m[n] = mx[n];
                    }
                    // (a row that has seen nothing keeps m = -inf and weights 2^(-inf) = 0; a NaN logit gives NaN)
                    const float mb = m[n] == -INFINITY ? 0.f : m[n] - kUp;
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float& p = s[n >> 1][j][2 * (n & 1) + e];
                            p = fast_exp2(p - mb);
                            sum += p;
                        }
                    l[n] = l[n] * alpha[n] + sum;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (__any_sync(0xFFFFFFFFu, alpha[n] != 1.f)) {   // columns 2c, 2c + 1 of the accumulator: rows 8 n + 2c, + 1
                        const float a0 = __shfl_sync(0xFFFFFFFFu, alpha[n], 8 * c), a1 = __shfl_sync(0xFFFFFFFFu, alpha[n], 8 * c + 4);
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            acc[n][i][0] *= a0; acc[n][i][1] *= a1; acc[n][i][2] *= a0; acc[n][i][3] *= a1;
                        }
                    }
                }
                // ---- out^T += V^T P^T
                uint32_t ph[NT][2][2], pl[NT][2][2];   // [rows][16 tokens][2]: weights as fp16 + residual
                auto weights = [&](int gi) {           // of scale group gi
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int j = 2 * k2 + h;
                            float v0 = 1.f, v1 = 1.f;
                            if (kScaled) {
                                const int gs = NG == 1 ? 0 : (gi * ng) >> 2;
                                const uint32_t at = sv + 4 * ((8 * j + 2 * c) * (NG == 1 ? 1 : ng) + gs);
                                v0 = ldsf(at);
                                v1 = ldsf(at + 4 * (NG == 1 ? 1 : ng));
                            }
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                float p0 = s[n >> 1][j][2 * (n & 1)], p1 = s[n >> 1][j][2 * (n & 1) + 1];
                                if (kScaled) {
                                    p0 *= v0;
                                    p1 *= v1;
                                    if (masked) {   // a hidden token's scale slot may hold anything
                                        if (!((word[n] >> (8 * j + 2 * c)) & 1u)) p0 = 0.f;
                                        if (!((word[n] >> (8 * j + 2 * c + 1)) & 1u)) p1 = 0.f;
                                    }
                                }
                                split2(p0, p1, ph[n][k2][h], pl[n][k2][h]);
                            }
                        }
                };
                if constexpr (NG == 1) weights(0);
                const int valid = sq.ctx - t0;   // rows from here on are not the sequence's
#pragma unroll
                for (int ch = 0; ch < CH; ++ch) {
                    uint32_t r[4];   // r[j]: bytes 2g, 2g + 1 of tokens 8j + 2c (low half) and 8j + 2c + 1
                    ldsm4_t(vt + chunk_off(ch), r);
                    uint32_t bad[4] = {0u, 0u, 0u, 0u};
                    bool any_bad = false;
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int u = 8 * j + 2 * c;
                            r[j] &= (u < valid ? 0x0000FFFFu : 0u) | (u + 1 < valid ? 0xFFFF0000u : 0u);
                            if constexpr (!kScaled) {   // NaN codes: 0 * NaN must not reach the rows that do not see them
                                bad[j] = FMT == E4M3 ? __vcmpeq4(r[j] & 0x7F7F7F7Fu, 0x7F7F7F7Fu)
                                                     : __vcmpgtu4(r[j] & 0x7F7F7F7Fu, 0x7B7B7B7Bu);
                                any_bad |= bad[j] != 0u;
                                r[j] &= ~bad[j];
                            }
                        }
                    }
                    auto pv = [&](int i, int k2, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_16816(acc[n][i], a0, a1, a2, a3, ph[n][k2][0], ph[n][k2][1]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_16816(acc[n][i], a0, a1, a2, a3, pl[n][k2][0], pl[n][k2][1]);
                    };
                    if constexpr (I4) {
#pragma unroll
                        for (int sub = 0; sub < SUB; ++sub) {
                            if constexpr (NG > 1) weights(SUB == 2 ? 2 * ch + sub : ch / CPG);
                            const bool mine = SUB == 1 || (g >> 2) == sub;   // channels 32 ch + 4g .. + 3
#pragma unroll
                            for (int k2 = 0; k2 < 2; ++k2) {
                                const uint32_t x = r[2 * k2] ^ 0x88888888u, y = r[2 * k2 + 1] ^ 0x88888888u;
#pragma unroll
                                for (int bb = 0; bb < 2; ++bb) {
                                    const uint32_t xs = bb ? x >> 8 : x, ys = bb ? y >> 8 : y;
                                    uint32_t a0 = nib_lo(xs), a1 = nib_hi(xs), a2 = nib_lo(ys), a3 = nib_hi(ys);
                                    if (!mine) a0 = a1 = a2 = a3 = 0u;
                                    pv(2 * ch + bb, k2, a0, a1, a2, a3);
                                }
                            }
                        }
                    } else {
                        if constexpr (NG > 1) {
                            if (ch % CPG == 0) weights(ch / CPG);
                        }
#pragma unroll
                        for (int k2 = 0; k2 < 2; ++k2) {
                            uint32_t a0, a1, a2, a3;   // channels 16 ch + 2g (a0, a2) and + 1 (a1, a3)
                            dec4<FMT>(prmt(r[2 * k2], 0u, 0x3120u), a0, a1);
                            dec4<FMT>(prmt(r[2 * k2 + 1], 0u, 0x3120u), a2, a3);
                            pv(ch, k2, a0, a1, a2, a3);
                        }
                        if constexpr (!kScaled) {
                            // channels whose V is NaN at a token a row does see: NaN, as the sum would be
                            if (masked && __any_sync(0xFFFFFFFFu, any_bad)) {
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    float hit[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                                    for (int k2 = 0; k2 < 2; ++k2) {
                                        uint32_t o[4], sees[2];   // 1.0 where V is NaN; 1.0 where row 8 n + g sees the token
#pragma unroll
                                        for (int h = 0; h < 2; ++h) {
                                            const uint32_t x = prmt(bad[2 * k2 + h], 0u, 0x3120u) & 0x3C3C3C3Cu;
                                            o[2 * h] = prmt(x, 0u, 0x1404u);       // byte 0, byte 1 as the high bytes of two halves
                                            o[2 * h + 1] = prmt(x, 0u, 0x3424u);
                                            const int u = 8 * (2 * k2 + h) + 2 * c;
                                            sees[h] = ((word[n] >> u) & 1u ? 0x3C00u : 0u) | ((word[n] >> (u + 1)) & 1u ? 0x3C000000u : 0u);
                                        }
                                        mma_16816(hit, o[0], o[1], o[2], o[3], sees[0], sees[1]);
                                    }
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        if (hit[e] > 0.f) acc[n][ch][e] = __int_as_float(0x7FC00000);
                                }
                            }
                        }
                    }
                }
            }
            __syncwarp();   // every lane has read the stage
            ++ck;
            cst = cst + 1 == kStages ? 0 : cst + 1;
            cph ^= cst == 0 ? 1u : 0u;
            if (!failed) issue_ready();
        }

        // ------------------------------------------------------ segment end ----
        const bool whole = seg == sw.n;
        const int slot = team * 2 + (sw.t == 0 ? 1 : 0);
        const float s_out = kScaled ? 1.0f : s_fp8;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            l[n] += __shfl_xor_sync(0xFFFFFFFFu, l[n], 1);
            l[n] += __shfl_xor_sync(0xFFFFFFFFu, l[n], 2);
        }
        if (solo) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (!whole && c == 0) ws_ml[(int64_t)slot * RT + 8 * n + g] = make_float2(m[n], l[n]);
                // 1 / sum of rows 8 n + 2c and + 1 (a row that saw nothing: 0)
                const float inv = l[n] == 0.f ? 0.f : s_out / l[n];
                const float w0 = __shfl_sync(0xFFFFFFFFu, inv, 8 * c), w1 = __shfl_sync(0xFFFFFFFFu, inv, 8 * c + 4);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * n + 2 * c + e;
                    if (r >= R) continue;
                    const float w = whole ? (e ? w1 : w0) : s_out;
                    uint16_t* od = a.out + out_row(r) * D;
                    float* pd = ws_acc + ((int64_t)slot * RT + r) * D;
                    if constexpr (I4) {
#pragma unroll
                        for (int ch = 0; ch < CH; ++ch) {
                            const float4 v = make_float4(acc[n][2 * ch][e] * w, acc[n][2 * ch][2 + e] * w,
                                                         acc[n][2 * ch + 1][e] * w, acc[n][2 * ch + 1][2 + e] * w);
                            const int d = 32 * ch + 4 * g;
                            if (whole) *reinterpret_cast<uint2*>(od + d) = make_uint2(pack_f16x2(v.x, v.y), pack_f16x2(v.z, v.w));
                            else *reinterpret_cast<float4*>(pd + d) = v;
                        }
                    } else {
#pragma unroll
                        for (int ch = 0; ch < CH; ++ch) {
                            const float2 v = make_float2(acc[n][ch][e] * w, acc[n][ch][2 + e] * w);
                            const int d = 16 * ch + 2 * g;
                            if (whole) *reinterpret_cast<uint32_t*>(od + d) = pack_f16x2(v.x, v.y);
                            else *reinterpret_cast<float2*>(pd + d) = v;
                        }
                    }
                }
            }
            __syncwarp();
        } else {
            if (c == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n) ml_s[warp * RT + 8 * n + g] = make_float2(m[n], l[n]);
            }
            __syncthreads();
            float fac[NT][2];   // 2^(m of this warp - m of the team) of rows 8 n + 2c, + 1
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * n + 2 * c + e;
                    float M = -INFINITY;
#pragma unroll
                    for (int w = 0; w < W; ++w) M = fmaxf(M, ml_s[w * RT + r].x);
                    fac[n][e] = fast_exp2(ml_s[warp * RT + r].x - (M == -INFINITY ? 0.f : M)) * s_out;
                }
            float* mine = merge + warp * RT * X::kMergeRow;
#pragma unroll
            for (int part = 0; part < D / 32; ++part) {   // 32 channels at a time
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float* dst = mine + (8 * n + 2 * c + e) * X::kMergeRow;
                        const float w = fac[n][e];
                        const int i = 2 * part;
                        if constexpr (I4) {
                            *reinterpret_cast<float4*>(dst + 4 * g) = make_float4(acc[n][i][e] * w, acc[n][i][2 + e] * w,
                                                                                  acc[n][i + 1][e] * w, acc[n][i + 1][2 + e] * w);
                        } else {
                            *reinterpret_cast<float2*>(dst + 2 * g) = make_float2(acc[n][i][e] * w, acc[n][i][2 + e] * w);
                            *reinterpret_cast<float2*>(dst + 16 + 2 * g) = make_float2(acc[n][i + 1][e] * w, acc[n][i + 1][2 + e] * w);
                        }
                    }
                __syncthreads();
                if (threadIdx.x < RT * 8) {   // a row's 4 channels per thread, the warps' sums in order
                    const int r = threadIdx.x >> 3, d = (threadIdx.x & 7) * 4;
                    float M = -INFINITY, sum = 0.f;
#pragma unroll
                    for (int w = 0; w < W; ++w) M = fmaxf(M, ml_s[w * RT + r].x);
                    const float Ms = M == -INFINITY ? 0.f : M;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const float2 x = ml_s[w * RT + r];
                        sum += x.y * fast_exp2(x.x - Ms);
                        const float4 y = *reinterpret_cast<const float4*>(merge + (w * RT + r) * X::kMergeRow + d);
                        v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
                    }
                    if (r < R) {
                        if (whole) {
                            const float inv = sum == 0.f ? 0.f : 1.0f / sum;
                            *reinterpret_cast<uint2*>(a.out + out_row(r) * D + 32 * part + d) =
                                make_uint2(pack_f16x2(v.x * inv, v.y * inv), pack_f16x2(v.z * inv, v.w * inv));
                        } else {
                            *reinterpret_cast<float4*>(ws_acc + ((int64_t)slot * RT + r) * D + 32 * part + d) = v;
                            if (part == 0 && d == 0) ws_ml[(int64_t)slot * RT + r] = make_float2(M, sum);
                        }
                    }
                }
                __syncthreads();   // before the buffer, the sums or Q are overwritten
            }
        }
        if (f + seg == hi && lead) {   // the last segment: parts of it that later teams hold
            int parts = 0;
            if (sw.t == 0 && !whole) {
                int left = sw.n - seg;
                for (int t = ct + 1; left > 0; ++t, ++parts) left -= len + (t < extra ? 1 : 0);
            }
            *hdr = make_int4(sw.b, sw.kvh, cls, parts);
        }
        f += seg;
        if (f < hi) {
            sw.t = 0;
            if (++sw.kvh == Hkv) {
                sw.kvh = 0;
                do { ++sw.b; } while (sw.b < B && S[sw.b + 1] == S[sw.b]);
                sw.n = S[sw.b + 1] - S[sw.b];
            }
        }
    }
}

// Merges the parts of a row tile that several teams hold: block (team, row
// group of 8), one warp per row: out = sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i
// over the team's slot 1 and the following teams' slots 0.
template <int D>
__global__ void __launch_bounds__(256) verify_reduce_kernel(const VerifyArgs a, const VerifyPlan plan) {
    griddep_wait();
    const int4 h = reinterpret_cast<const int4*>(a.ws)[blockIdx.x];
    if (h.w == 0) return;
    const int G = a.num_q_heads / a.cache.num_kv_heads, RT = plan.rows;
    const int r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const Seq sq = seq_of(a, h.x, false);
    const int rr = h.z * RT + r;
    if (rr >= sq.n * G) return;
    const float2* ml = reinterpret_cast<const float2*>(a.ws + verify_ml_off(plan.teams));
    const float* acc = reinterpret_cast<const float*>(a.ws + verify_acc_off(plan.teams, RT));
    auto slot = [&](int i) -> int64_t { return (int64_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0); };
    float M = -INFINITY;
    for (int i = lane; i <= h.w; i += 32) M = fmaxf(M, ml[slot(i) * RT + r].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, off));
    const float Ms = M == -INFINITY ? 0.f : M;
    constexpr int V = D / 32;
    float o[V], sum = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = 0.f;
#pragma unroll 4
    for (int i = 0; i <= h.w; ++i) {
        const float2 x = ml[slot(i) * RT + r];
        const float e = fast_exp2(x.x - Ms);
        sum += e * x.y;
        const float* src = acc + (slot(i) * RT + r) * D + V * lane;
        if constexpr (V == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            o[0] += e * v.x; o[1] += e * v.y; o[2] += e * v.z; o[3] += e * v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            o[0] += e * v.x; o[1] += e * v.y;
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    uint16_t* dst = a.out + ((int64_t)(sq.q0 + rr / G) * a.num_q_heads + h.y * G + rr % G) * D + V * lane;
    if constexpr (V == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_f16x2(o[0] * inv, o[1] * inv), pack_f16x2(o[2] * inv, o[3] * inv));
    else
        *reinterpret_cast<uint32_t*>(dst) = pack_f16x2(o[0] * inv, o[1] * inv);
}

// ---------------------------------------------------------------- host --

// 2-D view [rows][row bytes] of one code array; a row is one swizzle span.
inline bool make_tmap(CUtensorMap* m, void* base, int64_t rows, int rb, int box_rows) {
    static PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)rb, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)rb};
    cuuint32_t box[2] = {(cuuint32_t)rb, (cuuint32_t)box_rows}, estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               rb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : (rb == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B),
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT, int D, int RT, int NG>
cudaError_t launch_t(const CUtensorMap& tk, const CUtensorMap& tv, const VerifyArgs& a, const VerifyPlan& p, cudaStream_t s) {
    using X = Shape<FMT, D, RT>;
    auto kern = verify_kernel<FMT, D, RT, NG>;
    const int smem = Layout(X::kWarps, X::kTileBytes, X::kTeamBytes, X::kScaled, a.cache.ngroups, a.batch).total + 1024;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = once_per_device(done, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    Layout(X::kWarps, X::kTileBytes, X::kTeamBytes, X::kScaled, 4, 4096).total + 1024);
    });
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3((unsigned)p.ctas), dim3(X::kThreads), smem, s, tk, tv, a, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(verify_reduce_kernel<D>, dim3((unsigned)p.teams, (unsigned)(RT / 8)), dim3(256), 0, s, a, p);
}

template <int FMT, int D, int NG>
cudaError_t launch_rt(const CUtensorMap& tk, const CUtensorMap& tv, const VerifyArgs& a, const VerifyPlan& p, cudaStream_t s) {
    if (p.rows == 8) return launch_t<FMT, D, 8, NG>(tk, tv, a, p, s);
    if (p.rows == 16) return launch_t<FMT, D, 16, NG>(tk, tv, a, p, s);
    return launch_t<FMT, D, 32, NG>(tk, tv, a, p, s);
}

// One format's kernels (one translation unit each).
template <int FMT>
cudaError_t launch_fmt(const VerifyArgs& a, const VerifyPlan& p, cudaStream_t s) {
    const int rb = row_bytes(FMT, a.cache.head_dim), box = a.cache.block_size >= kTile ? kTile : kBox;
    const int64_t rows = (int64_t)a.cache.num_blocks * a.cache.num_kv_heads * a.cache.block_size;
    CUtensorMap tk, tv;
    if (!make_tmap(&tk, a.cache.k_codes, rows, rb, box) || !make_tmap(&tv, a.cache.v_codes, rows, rb, box))
        return cudaErrorInvalidValue;
    if constexpr (FMT == INT8 || FMT == INT4) {
        if (a.cache.ngroups > 1)
            return a.cache.head_dim == 64 ? launch_rt<FMT, 64, 4>(tk, tv, a, p, s) : launch_rt<FMT, 128, 4>(tk, tv, a, p, s);
    }
    return a.cache.head_dim == 64 ? launch_rt<FMT, 64, 1>(tk, tv, a, p, s) : launch_rt<FMT, 128, 1>(tk, tv, a, p, s);
}

cudaError_t launch_e4m3(const VerifyArgs& a, const VerifyPlan& p, cudaStream_t s);
cudaError_t launch_e5m2(const VerifyArgs& a, const VerifyPlan& p, cudaStream_t s);
cudaError_t launch_int8(const VerifyArgs& a, const VerifyPlan& p, cudaStream_t s);
cudaError_t launch_int4(const VerifyArgs& a, const VerifyPlan& p, cudaStream_t s);

}  // namespace verify
}  // namespace kvq
