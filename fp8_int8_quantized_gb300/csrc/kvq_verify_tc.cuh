// Attention of a short chunk of new tokens over the paged quantized cache on
// the fifth-generation tensor cores (tcgen05), for head_dim 128 (the formulas
// and the cut into ranges, segments and partials are those of kvq_verify.cuh).
//
// The tokens are the M side of both products, so that a tile costs the same
// whatever the number of rows: per tile of 128 tokens
//   S^T [128 tokens][RT]  = K [128][D] . Q^T [D][RT]          8 MMAs of N = RT
//   O^T [D][2 RT]        += V^T [D][128] . [P_hi | P_lo]      8 MMAs of N = 2 RT
// with P = P_hi + P_lo in fp16 pairs (~22 bits) side by side as columns, summed
// when the accumulator is read: V is read once for both.  (The rows as M, 128
// of them whatever the chunk, would cost four times the products at 32 rows.)
// P carries the token's own V scale, and a row's running maximum is that of the
// weight with it (log2_scale in kvq_verify.cuh).
//
// Roles of the CTA's 20 warps (one CTA per SM; registers moved between the
// warpgroups with setmaxnreg):
//   * warps 8-11 and 12-15 (dequant, of the even and of the odd tiles): a warp
//     copies the codes of its 32 tokens through the block table into a ring of
//     its own (cp.async, 16 bytes per lane, so no other warp waits for them; TMA
//     boxes of 16 rows cost an issuing warp ~100 cycles each, 16 per tile); then
//     a thread is a token: exact conversion to fp16; K into tensor memory as the
//     A operand of S (it never returns to shared memory, whose bandwidth is the
//     next limit after HBM's), V into the 128-byte-swizzled layout of an MN-major
//     A operand (tokens past the context as zeros).  With group scales V is
//     stored as code x scale in an fp16 pair of tiles (value, residual), by three
//     fp16 FMAs per pair of channels (through fp32 it took eight: 460 -> 414 us
//     in the last case below); its scales come through the ring as well;
//   * warps 16 and 17 (MMA): S, and O += P V (one warp for both met six waits
//     and 16 MMAs per tile in turn and was the slowest role);
//   * warp 18: the segment's Q (asynchronous copies of all rows at once);
//   * warps 0-3 and 4-7 (softmax): one stream each of the even and odd tiles,
//     with a maximum, sums and an O accumulator of its own, joined at the end of
//     a segment.  A thread is a token: its RT logits take its own K scale,
//     its weights its own V scale, and the rows' maxima come from shared memory.
//     A tile whose logits stay within 2^kLazy of the rows' maxima needs no
//     maximum at all (one vote); else the maxima are taken across the lanes and
//     O is rescaled.  With group scales (NG 4) S is one product per scale group
//     and the thread adds them up with its token's scales.
// Every wait is bounded (2 s); after a timeout every role runs to its end
// without waiting, and the copies and MMAs in flight are drained.
//
// What bounds it: the roles, one or two warps per scheduler each, at 4 to 6 cycles
// per instruction of a warp; a tile of 128 tokens takes ~1800 cycles (16 or 32
// rows), ~2070 (64 rows), ~2600 (group scales, 32 rows), and HBM's share of it
// is ~1400 (8-bit codes).  Measured, the reduction included, calls back to back
// over three sets of inputs (the first after a flush of L2):
//   E4M3, 32 x 8192 tokens, 64 / 8 heads, 4 queries (32 rows)       101 us, 5.4 TB/s (115)
//   E5M2, 24 x 515 .. 8191, 32 / 8 heads, trees of 9 .. 16 (64)      82 us, 2.7 TB/s (88)
//   INT8, 16 x 4096, 40 / 40 heads, 8 queries (16)                  122 us, 5.7 TB/s (137)
//   INT4, 32-channel groups, 3 x ~115000, 64 / 8, 5 .. 7 (2 x 32)   343 us, 1.29 TB/s
//   INT4, a scale per row, 32 x 8192, 64 / 8, 4 (32)                123 us, 2.4 TB/s
//   E5M2, one sequence of 1000, 32 / 8, 4 queries (16)               (17 us)
#pragma once

#include <type_traits>

#include "kvq_verify.cuh"

namespace kvq {
namespace verify {
namespace tc {

constexpr int kTok = 128;          // tokens per tile
constexpr int D = 128;
constexpr int kDqWarp = 8, kMmaWarp = 16, kQWarp = 18;   // 16: S, 17: P V
constexpr int kThreads = 640;
// Registers per thread: 96 at launch (640 x 96 = 61440), then 136 for the two
// softmax warpgroups, 72 for the two of dequant, 64 for the rest: 128 x (2 x 136 + 2 x 72 + 64) = 61440.
constexpr int kLaunchRegs = 96;
constexpr uint32_t kBlk = kTok * 128;       // one 64-column block of a K, V or P tile
constexpr uint32_t kTileV = 2 * kBlk;       // fp16 V tile
constexpr int kMaxBatch = kMaxTcBatch;
constexpr float kNone = -1e30f;             // the maximum of a row that has seen nothing

// Byte offset of (row, 16-byte chunk) in a [rows][128 B] block with the 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128(uint32_t row, uint32_t chunk) {
    return (row >> 3) * 1024u + (row & 7u) * 128u + ((chunk ^ (row & 7u)) << 4);
}
// Shared-memory matrix descriptor (version 1, 128-byte swizzle).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
           (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// kind::f16, fp32 accumulator, f16 A and B; a_mn / b_mn: MN-major operands.
__host__ __device__ constexpr uint32_t idesc(uint32_t m, uint32_t n, uint32_t a_mn, uint32_t b_mn) {
    return (1u << 4) | (a_mn << 15) | (b_mn << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
// One lane of a converged warp, the same every time.  (The warp index, the
// addresses and this choice are warp-uniform to the compiler, so the operands
// stay in uniform registers: ~48 cycles per MMA of N = 64 against ~200 when
// a branch on the lane number issues them.)
__device__ __forceinline__ bool elect() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(e));
    return e != 0;
}
// Issued by that lane; A from shared or tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t ad, uint64_t bd, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(ad), "l"(bd), "r"(id), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t at, uint64_t bd, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(at), "l"(bd), "r"(id), "r"(accumulate)
        : "memory");
}
// Arrive once on `bar` when every MMA this thread issued so far is done.
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 16 consecutive 32-bit columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t t, float* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(t));
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const float* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
        "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]),
        "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
        : "memory");
}
// After wait_ld: no use of the loaded registers is scheduled before it.
__device__ __forceinline__ void reg_fence16(float* r) {
    asm volatile("" : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                      "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]));
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// One attempt that may sleep in the barrier for up to 10 us (a polling loop of
// the waiting warps took half of the issue slots).
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity), "r"(10000) : "memory");
    return ok != 0;
}
// Barrier of `n` threads that also says whether any of them passes true.
__device__ __forceinline__ bool bar_any(int id, int n, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %3, 0;\n\tbarrier.cta.red.or.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r) : "r"(id), "r"(n), "r"((int)v) : "memory");
    return r != 0;
}

// fp16 pair of p0 - h.lo, p1 - h.hi (a mixed-precision FMA each: exact product, one rounding).
__device__ __forceinline__ uint32_t residual(uint32_t h, float p0, float p1) {
    uint32_t r;
    asm("{\n\t.reg .f16 a, b, m1;\n\t.reg .f32 r0, r1;\n\tmov.b32 {a, b}, %1;\n\tmov.b16 m1, 0xBC00;\n\t"
        "fma.rn.f32.f16 r0, a, m1, %2;\n\tfma.rn.f32.f16 r1, b, m1, %3;\n\tcvt.rn.f16x2.f32 %0, r1, r0;\n\t}"
        : "=r"(r) : "r"(h), "f"(p0), "f"(p1));
    return r;
}
// h (codes in fp16) times the scale s1 + s2 as an fp16 pair: hi = rn(h s1), lw = rn(h s2 + (h s1 - hi)).
// The difference is exact (a rounding error of a product), so hi + lw is h (s1 + s2) to 2^-22.
__device__ __forceinline__ void scale_pair(uint32_t h, uint32_t s1, uint32_t s2, uint32_t& hi, uint32_t& lw) {
    asm("{\n\t.reg .b32 e, n;\n\tmul.rn.f16x2 %0, %2, %3;\n\tneg.f16x2 n, %0;\n\tfma.rn.f16x2 e, %2, %3, n;\n\t"
        "fma.rn.f16x2 %1, %2, %4, e;\n\t}"
        : "=&r"(hi), "=r"(lw) : "r"(h), "r"(s1), "r"(s2));
}
// INT4 nibbles as nib_lo / nib_hi give them, times 2^-2; INT8 codes times 2^-6: below 2 in
// magnitude, so that the scale's terms (times 2^2, 2^6) stay in fp16's normal range as long as V does.
__device__ __forceinline__ uint32_t nib_lo4(uint32_t x) {   // (1024 + n) / 4 - 258
    return hfma2_const((x & 0x000F000Fu) | 0x64006400u, 0x34003400u, 0xDC08DC08u);
}
__device__ __forceinline__ uint32_t nib_hi4(uint32_t x) {   // (1024 + 16 n) / 64 - 18
    return hfma2_const((x & 0x00F000F0u) | 0x64006400u, 0x24002400u, 0xCC80CC80u);
}
__device__ __forceinline__ void byte4_64(uint32_t w, uint32_t& lo, uint32_t& hi) {   // (1024 + 128 + code) / 64 - 18
    const uint32_t x = w ^ 0x80808080u;
    lo = hfma2_const(prmt(x, 0x64646464u, 0x4140u), 0x24002400u, 0xCC80CC80u);
    hi = hfma2_const(prmt(x, 0x64646464u, 0x4342u), 0x24002400u, 0xCC80CC80u);
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

enum Bar : int {
    KFULL0, KFULL1,   // dequant -> MMA: K in tensor memory (128)
    KFREE0, KFREE1,   // MMA -> dequant (commit of S)
    VFULL0, VFULL1,   // dequant -> MMA (128)
    VFREE0, VFREE1,   // MMA -> dequant, softmax (commit of P V): V, P free, O up to date
    PFULL0, PFULL1,   // softmax -> MMA: P stored (128)
    SFULL0,           // MMA -> softmax of the stream, per S buffer (commit)
    SFREE0 = SFULL0 + 4,   // softmax -> MMA: S read, per S buffer (128)
    SFREE3 = SFREE0 + 3,
    QFULL0, QFULL1,   // Q warp -> MMA: Q of segment s in its buffer, barrier s % 2 (32)
    QFREE0, QFREE1,   // MMA -> Q warp: every S of segment s done (commit)
    OFREE,            // softmax -> MMA: both O accumulators read, once per segment (256)
    OFINAL,           // every MMA done (commits of both MMA warps)
    kNumBars
};

template <int FMT, int RT, int NG>
struct Smem {
    static constexpr uint32_t kUnit = kTok * row_bytes(FMT, D);             // codes of K or of V of a tile
    static constexpr uint32_t kGroups = NG > 1 ? kTok * 16 : 0;             // V's group scales of a tile
    static constexpr uint32_t kVBuf = kTileV * (NG > 1 ? 2 : 1);            // V, or value and residual
    static constexpr int kQBufs = RT == 64 ? 1 : 2;
    static constexpr uint32_t kPBlocks = RT == 64 ? 2 : 1;                  // P tile: [128][2 RT] in 64-column blocks
    static constexpr uint32_t kV = 0, kP = 2 * kVBuf;
    static constexpr uint32_t kQ = kP + 2 * kPBlocks * kBlk;                // [RT][128] in two 64-column blocks
    static constexpr uint32_t kStage = kQ + kQBufs * RT * 256;
    // code units per dequant warpgroup (every second one a V's, with its group scales apart): as
    // many as fit beside the statistics, the scan of kMaxBatch and the static arrays
    static constexpr uint32_t ring(int units) { return units * kUnit + (units + 1) / 2 * kGroups; }
    static constexpr int fit(int units) {
        return units <= 1 || kStage + 2 * ring(units) + 21 * RT * 4 + (2 * kMaxBatch + 1) * 4 + 512 + 2048 <= 227 * 1024 ? units : fit(units - 1);
    }
    static constexpr int kUnits = fit(6), kVUnits = (kUnits + 1) / 2;
    static constexpr uint32_t kM = kStage + 2 * ring(kUnits);          // f32 [stream][RT]: maxima
    static constexpr uint32_t kMx = kM + 2 * RT * 4;                   // f32 [stream][warp][RT]: a tile's maxima
    static constexpr uint32_t kL = kMx + 8 * RT * 4;                   // f32 [stream][warp][RT]: sums
    static constexpr uint32_t kF = kL + 8 * RT * 4;                    // f32 [stream][RT]: rescaling factors
    static constexpr uint32_t kRow = kF + 2 * RT * 4;                  // int [RT]: the rows' places in the output
    static constexpr uint32_t kBar = kRow + RT * 4;
    static constexpr uint32_t kTmemSlot = kBar + kNumBars * 8;
    static constexpr uint32_t kAbort = kTmemSlot + 4;
    // NaN codes or scales met in segment s, in slot s % kSlots, which the end of segment s - kSlots has to have
    // reset before.  A code of tile j is noted once P V of tile j - 2 is done, so segment s - 3 has ended:
    // 4 slots.  A scale is noted before that wait, when P V of tile j - 4 is and segment s - 5 has ended: 8
    // (4 slots and the note kept until after the wait: 354 us in the INT4 case above, with 8 344).
    static constexpr int kSlots = NG > 1 ? 8 : 4;
    static constexpr uint32_t kNan = kAbort + 4;                       // int [kSlots]
    static constexpr uint32_t kScan = kNan + 4 * kSlots;               // int S[B + 1], context lengths [B]
    static constexpr uint32_t bytes(int B) { return kScan + (2 * B + 1) * 4 + 1024; }
    static_assert(kUnits >= 1 && bytes(kMaxBatch) + 512 <= 227 * 1024, "shared memory of one CTA");
};

// The tiles lo .. lo + cnt - 1 of its class's flat list are a CTA's.  Every CTA
// gets as much work, counting the first tile of a pair as 1 + kSegTiles: a
// segment costs that much more than its tiles (the pipeline runs empty, O is
// read and written).  With equal numbers of tiles a CTA of short sequences
// worked twice as long as one of long ones: 24 sequences of 515 .. 8191 tokens,
// 32 / 8 heads, chunks of 9 .. 16: 115 us (L2 flushed), with a weight of 2: 98, of
// 4: 88, of 6: 86; 32 x 8192 tokens: 117, 115, 115, 117.  A CTA with few tiles counts them
// alone (and skips the scan: 2 us of a small call).
constexpr uint32_t kSegTiles = 4;
struct Share {
    int lo, cnt;
    int parts;   // CTAs after this one that hold tiles of the pair this share ends inside of
};
struct Cut {     // units of work 0 .. U - 1 over the class's CTAs
    uint32_t len, extra;
    __device__ __forceinline__ Cut(uint32_t U, uint32_t ctas) : len(U / ctas), extra(U % ctas) {}
    __device__ __forceinline__ uint32_t first(uint32_t cta) const { return cta * len + min(cta, extra); }
    __device__ __forceinline__ uint32_t cta_of(uint32_t u) const {
        return u < extra * (len + 1) ? u / (len + 1) : extra + (u - extra * (len + 1)) / len;
    }
};
// Called by all threads.  (Units fit 32 bits: the host bounds the tiles by 2^29.)
__device__ __forceinline__ Share share_of(const int* S, int B, int Hkv, uint32_t ctas, uint32_t cta) {
    __shared__ int wsum[kThreads / 32], out[3];
    const uint32_t T = ctas ? Hkv * S[B] : 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (T == 0) return Share{0, 0, 0};   // the same for every thread
    const uint32_t wt = min(kSegTiles, T / ctas / 8);
    if (wt == 0) {
        const Cut c(T, ctas);
        const uint32_t u0 = c.first(cta), u1 = c.first(cta + 1);
        int parts = 0;
        if (u1 > u0 && u1 < T) {
            const Walk w = locate(S, B, Hkv, u1 - 1);   // the share's last tile
            if (w.t + 1 < w.n) parts = c.cta_of(u1 - 1 + w.n - 1 - w.t) - cta;
        }
        return Share{(int)u0, (int)(u1 - u0), parts};
    }
    // sequences with tiles before this thread's
    const int per = (B + kThreads - 1) / kThreads;
    const int b0 = min(B, (int)threadIdx.x * per), b1 = min(B, b0 + per);
    int live = 0;
    for (int b = b0; b < b1; ++b) live += S[b + 1] > S[b];
    int x = live;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    int before = x - live, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += wsum[w];
        all += wsum[w];
    }
    const uint32_t U = T + wt * Hkv * all;
    const Cut c(U, ctas);
    const uint32_t u0 = c.first(cta), u1 = c.first(cta + 1);
    if (threadIdx.x == 0) {   // (an end behind the last unit lies in no sequence)
        if (u0 == U) out[0] = T;
        if (u1 == U) out[1] = T, out[2] = 0;
    }
    for (int b = b0; b < b1; ++b) {
        const uint32_t n = S[b + 1] - S[b];
        if (n == 0) continue;
        const uint32_t base = Hkv * (S[b] + wt * before), end = base + Hkv * (n + wt);
        ++before;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t u = e ? u1 : u0;
            if (u < base || u >= end) continue;
            const uint32_t kvh = (u - base) / (n + wt), t = (u - base) % (n + wt);   // its first wt units: no tile
            out[e] = Hkv * S[b] + kvh * n + (t > wt ? t - wt : 0);
            if (e) out[2] = t > wt ? c.cta_of(base + (kvh + 1) * (n + wt) - 1) - cta : 0;
        }
    }
    __syncthreads();
    return Share{out[0], out[1] - out[0], out[2]};
}

template <int FMT, int RT, int NG>
__global__ void __launch_bounds__(kThreads, 1)
    verify_tc_kernel(const VerifyArgs a, const VerifyPlan plan) {
    using L = Smem<FMT, RT, NG>;
    constexpr bool I4 = FMT == INT4, kScaled = FMT == INT8 || FMT == INT4;
    constexpr int RB = row_bytes(FMT, D), NU = L::kUnits, kSlots = L::kSlots;
    // tensor memory: K 2 x 64 columns (fp16 pairs), O 2 x 2 RT, and S in two buffers per stream where
    // they fit (S of the stream's next tile then runs under the softmax of this one), NG x RT each
    constexpr int SB = 128 + 4 * NG * RT + 4 * RT <= 512 ? 4 : 2;   // S of tile j: buffer j % SB
    constexpr uint32_t kColS = 128, kColO = kColS + SB * NG * RT, kUsed = kColO + 4 * RT;
    constexpr int kLogSB = SB == 4 ? 2 : 1;
    constexpr uint32_t kCols = kUsed <= 256 ? 256 : 512;
    static_assert(kUsed <= 512, "tensor memory");
    constexpr uint32_t kIdS = idesc(128, RT, 0, 0), kIdO = idesc(128, 2 * RT, 1, 1), kIdLo = idesc(128, RT, 1, 1);
    constexpr float kScaleUp = I4 ? 4.f : 64.f, kMaxScale = 65504.f / kScaleUp;   // V's group scales
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = __shfl_sync(0xFFFFFFFFu, smem_u32(sm), 0);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::kBar);
    volatile int* abort = reinterpret_cast<volatile int*>(sm + L::kAbort);
    volatile int* nan_seen = reinterpret_cast<volatile int*>(sm + L::kNan);
    int* S = reinterpret_cast<int*>(sm + L::kScan);
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const int B = a.batch, Hkv = a.cache.num_kv_heads, BS = a.cache.block_size, G = a.num_q_heads / Hkv;
    const int ng = a.cache.ngroups;
    int4* hdr = reinterpret_cast<int4*>(a.ws) + blockIdx.x;
    if (tid == 0) {
        for (int i = 0; i < kNumBars; ++i) {
            const bool c128 = i == KFULL0 || i == KFULL1 || i == VFULL0 || i == VFULL1 || i == PFULL0 || i == PFULL1 || (i >= SFREE0 && i <= SFREE3);
            mbar_init(&bars[i], c128 ? 128u : i == QFULL0 || i == QFULL1 ? 32u : i == OFREE ? 256u : i == OFINAL ? 2u : 1u);
        }
        *abort = 0;
        for (int i = 0; i < kSlots; ++i) nan_seen[i] = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + L::kTmemSlot), "r"(kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    griddep_wait();     // the inputs may come from the previous kernel
    griddep_launch();
    fence_before();
    int* ctx_s = S + B + 1;
    for (int b = tid; b < B; b += kThreads) ctx_s[b] = __ldg(a.context_lens + b);
    const ClassOf co = scan_class<kThreads, kTok>(a, plan.row_tiles, RT, S);   // syncs the CTA
    fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *reinterpret_cast<uint32_t*>(sm + L::kTmemSlot), 0);
    const int cls = co.cls;
    const Share sh = share_of(S, B, Hkv, cls < 0 ? 0 : co.ctas, co.cta);   // syncs the CTA
    // this CTA's tiles: lo .. lo + cnt - 1
    const int lo = sh.lo, cnt = __shfl_sync(0xFFFFFFFFu, sh.cnt, 0);

    // Waits that give up for the whole CTA at once.
    auto wait = [&](int bar, uint32_t parity) -> bool {
        const uint32_t at = sb + L::kBar + 8 * bar;
        bool ok = try_wait(at, parity);
        if (__all_sync(0xFFFFFFFFu, ok)) return true;
        for (const uint64_t t0 = globaltimer_ns(); !ok && !*abort; ok = try_wait(at, parity)) {
            if (globaltimer_ns() - t0 > kWaitLimitNs) {
                record_error(a.err, DEV_ERR_TIMEOUT, bar);   // (the first one is kept)
                *abort = 1;
            }
        }
        return __all_sync(0xFFFFFFFFu, ok);   // the warp goes on as one
    };
    auto next_pair = [&](Walk& w) {   // the pair after w's
        w.t = 0;
        if (++w.kvh == Hkv) {
            w.kvh = 0;
            do { ++w.b; } while (w.b < B && S[w.b + 1] == S[w.b]);
            w.n = w.b < B ? S[w.b + 1] - S[w.b] : 1;
        }
    };

    if (cnt == 0) {
        if (tid == 0) *hdr = make_int4(0, 0, 0, 0);
    } else if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == kQWarp) {
            // ------------------------------------------------------------ Q ----
            Walk qw = locate(S, B, Hkv, lo);
            const int qc = lane & 15;   // this lane's 16-byte chunk of the rows lane / 16, + 2, ...
#pragma unroll 1
            for (int qs = 0, qj = 0; qj < cnt; ++qs) {
                const Seq sq = seq_of<kTok>(a, qw.b, false);
                const int R = min(RT, sq.n * G - cls * RT);
                // the buffer is free once every S of the segment that used it is done
                const int prev = qs - L::kQBufs;
                if (prev >= 0 && !wait(QFREE0 + (prev & 1), (prev >> 1) & 1)) break;
                const uint32_t qb = sb + L::kQ + (L::kQBufs == 2 ? (qs & 1) * RT * 256 : 0) + (qc >> 3) * (RT * 128);
                int qi = (cls * RT + (lane >> 4)) / G, h = (cls * RT + (lane >> 4)) % G;
#pragma unroll 4
                for (int r = lane >> 4; r < RT; r += 2) {   // all rows in flight at once; zeros behind the last
                    const uint16_t* src = a.q + ((int64_t)(sq.q0 + (r < R ? qi : 0)) * a.num_q_heads + qw.kvh * G + h) * D + qc * 8;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(qb + sw128(r, qc & 7)), "l"(src), "r"(r < R ? 16 : 0) : "memory");
                    h += 2;
                    while (h >= G) { h -= G; ++qi; }
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                if (I4) {   // the channel order of the codes, of this lane's own chunks
#pragma unroll 4
                    for (int r = lane >> 4; r < RT; r += 2) {
                        const uint32_t at = qb + sw128(r, qc & 7);
                        const uint4 x = lds128(at);
                        sts128(at, prmt(x.x, x.z, 0x5410u), prmt(x.x, x.z, 0x7632u), prmt(x.y, x.w, 0x5410u), prmt(x.y, x.w, 0x7632u));
                    }
                }
                fence_async();
                mbar_arrive(&bars[QFULL0 + (qs & 1)]);
                qj += min(cnt - qj, qw.n - qw.t);
                next_pair(qw);
            }
        } else if (warp < kQWarp) {
            // ---------------------------------------------------------- MMA ----
            Walk w = locate(S, B, Hkv, lo);
            auto uni = [](int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); };   // (uniform to the compiler too)
            int seg = 0, js = 0, je = uni(min(cnt, w.n - w.t));                // the segment's tiles js .. je - 1
            auto next_seg = [&](int j) {
                ++seg;
                js = j;
                next_pair(w);
                je = uni(min(cnt, j + w.n));
            };
            if (warp == kMmaWarp) {   // S
                const uint64_t dq0 = smem_desc(sb + L::kQ, 16, 1024);
                bool ok = wait(QFULL0, 0);
#pragma unroll 1
                for (int j = 0; j < cnt && ok; ++j) {
                    const int sl = j & 1;
                    if (j == je) {
                        next_seg(j);
                        ok = wait(QFULL0 + (seg & 1), (seg >> 1) & 1);
                    }
                    const int sx = j & (SB - 1);
                    if (j >= SB) ok = ok && wait(SFREE0 + sx, ((j - SB) >> kLogSB) & 1);   // S of tile j - SB has been read
                    if (!ok || !wait(KFULL0 + sl, (j >> 1) & 1)) break;             // (a warp's lanes agree)
                    fence_after();
                    if (elect()) {
                        const uint64_t dq = dq0 + (((L::kQBufs == 2 ? seg & 1 : 0) * RT * 256) >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const int gi = kk / (8 / NG);   // scale group of these 16 channels
                            mma_ts(tmem + kColS + (sx * NG + gi) * RT, tmem + sl * 64 + kk * 8,
                                   dq + (((kk >> 2) * (RT * 128) + (kk & 3) * 32) >> 4), kIdS, kk % (8 / NG) > 0);
                        }
                        commit(&bars[SFULL0 + sx]);
                        commit(&bars[KFREE0 + sl]);
                        if (j + 1 == je) commit(&bars[QFREE0 + (seg & 1)]);
                    }
                    __syncwarp();
                }
            } else {                  // O += P V
                const uint64_t dv0 = smem_desc(sb + L::kV, kBlk, 1024), dp0 = smem_desc(sb + L::kP, kBlk, 1024);
                bool ok = true;
#pragma unroll 1
                for (int j = 0; j < cnt; ++j) {
                    const int sl = j & 1;
                    if (j == je) {
                        next_seg(j);
                        ok = wait(OFREE, (seg - 1) & 1);
                    }
                    if (!ok || !wait(VFULL0 + sl, (j >> 1) & 1) || !wait(PFULL0 + sl, (j >> 1) & 1)) break;
                    fence_after();
                    if (elect()) {
                        const uint32_t o = tmem + kColO + sl * 2 * RT;
                        uint64_t dv = dv0 + ((sl * L::kVBuf) >> 4), dp = dp0 + ((sl * L::kPBlocks * kBlk) >> 4);
#pragma unroll
                        for (int kk = 0; kk < kTok / 16; ++kk, dv += 2048 >> 4, dp += 2048 >> 4) {
                            mma_ss(o, dv, dp, kIdO, j - js >= 2 || kk > 0);
                            // V's residual times P's value, to the columns of P's residual: a sum of small terms rounds
                            // less, and the values' columns take half as many additions
                            if (NG > 1) mma_ss(o + RT, dv + (kTileV >> 4), dp, kIdLo, 1u);
                        }
                        commit(&bars[VFREE0 + sl]);
                    }
                    __syncwarp();
                }
            }
            if (elect()) commit(&bars[OFINAL]);
        }
    } else if (warp >= kDqWarp) {
        // ---------------------------------------------------------- dequant ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const int sl = (warp - kDqWarp) >> 2;   // the tiles j with j % 2 = sl, and their buffers
        const int tok = tid & 127, lbs = 31 - __clz(BS);
        const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t sw = RB == 128 ? (tok & 7) : ((tok >> 1) & 3);   // the stage's swizzle of this row
        // ---- copies: units K, V of this warpgroup's tiles in turn; a warp copies its own 32 tokens.
        // Lane l looks up half l % 2 (16 tokens) of the warp's share of the window's tile l / 2,
        // 16 tiles of this warpgroup at a time, the block ids one window ahead.
        int win = sl;           // first tile of the window looked up next
        int wid = 0, woff = -1; // its block id and place in the block; -1: past the context or the range
        auto look_up = [&]() {
            const int j = win + 2 * (lane >> 1);
            woff = -1;
            if (j < cnt) {
                const Walk x = locate(S, B, Hkv, lo + j);
                const int t = x.t * kTok + (warp & 3) * 32 + (lane & 1) * 16;
                if (t < ctx_s[x.b]) {
                    wid = __ldg(a.block_tables + (int64_t)x.b * a.max_blocks_per_seq + (t >> lbs));
                    woff = x.kvh * BS + (t & (BS - 1));
                }
            }
            win += 32;
        };
        int wrow = -1;          // row in the code arrays (below 2^31) of this lane's half, -1: none
        auto next_window = [&]() {
            wrow = woff < 0 ? -1 : wid * (Hkv * BS) + woff;
            if (woff >= 0 && (unsigned)wid >= (unsigned)a.cache.num_blocks) {
                record_error(a.err, DEV_ERR_RANGE, wid);   // its rows count as zeros
                wrow = -1;
            }
            look_up();
        };
        look_up();
        next_window();
        int wk = 0;             // tile of the window that is copied next
        constexpr int LPR = RB / 16, RPI = 32 / LPR;   // lanes per row, rows per copy of a warp
        const int crow = lane / LPR, cch = lane % LPR;
        const uint32_t ring = sb + L::kStage + sl * L::ring(NU) + (warp & 3) * 32 * RB;
        const uint32_t cdst = ring + crow * RB + ((cch ^ (RB == 128 ? crow & 7 : (crow >> 1) & 3)) << 4);
        // this token's group scales of the V copied and of the V read next
        [[maybe_unused]] const uint32_t gring = sb + L::kStage + sl * L::ring(NU) + NU * L::kUnit + tok * 16;
        [[maybe_unused]] int gc = 0, gr = 0;
        int cu = 0;             // unit copied into next
        int krow[2] = {-1, -1};   // the two halves' rows in the code arrays, for V's copies after K's
        auto copy_unit = [&](const uint8_t* codes, [[maybe_unused]] bool is_v) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const bool have = krow[hf] >= 0;
                const uint8_t* src = codes + (have ? krow[hf] : 0) * (int64_t)RB + lane * 16;   // row crow, chunk cch
                const int n = have ? 16 : 0;   // else zeros
#pragma unroll
                for (int i = 0; i < 16 / RPI; ++i) {
                    // row hf * 16 + i * RPI + crow of the warp's 32: its swizzle is crow's, and
                    // the odd copies' (rows 4 further) with the upper bit flipped
                    const uint32_t dst = cdst + cu * L::kUnit + (hf * 16 + i * RPI) * RB;
                    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(RB == 128 && (i & 1) ? dst ^ 64u : dst),
                                 "l"(src + i * RPI * RB), "r"(n) : "memory");
                }
            }
            if constexpr (NG > 1) {
                if (is_v) {   // lane l's token's scales
                    const int r = lane < 16 ? krow[0] : krow[1];
                    const float* src = a.cache.v_scales + (r < 0 ? 0 : r + (lane & 15)) * (int64_t)ng;
                    const uint32_t dst = gring + gc * L::kGroups;
                    if (++gc == L::kVUnits) gc = 0;
                    if (ng == 4) asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(r < 0 ? 0 : 16) : "memory");
                    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(r < 0 ? 0 : 8) : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (++cu == NU) cu = 0;
        };
        bool k_next = true;     // the unit copied next is a K
        auto copy_next = [&]() {
            if (k_next) {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) krow[hf] = __shfl_sync(0xFFFFFFFFu, wrow, 2 * wk + hf);
                if (++wk == 16) {
                    wk = 0;
                    next_window();
                }
            }
            copy_unit(k_next ? a.cache.k_codes : a.cache.v_codes, !k_next);
            k_next = !k_next;
        };
#pragma unroll 1
        for (int i = 0; i < NU; ++i) copy_next();
        int ru = 0;             // unit read next
        auto landed = [&]() {
            asm volatile("cp.async.wait_group %0;" ::"n"(NU - 1) : "memory");
            __syncwarp();
        };
        auto read_done = [&]() {   // the unit is free: the next one into it
            __syncwarp();
            copy_next();
            if (++ru == NU) ru = 0;
        };
        // the segment's tiles js .. je - 1, its context and first draft position; this thread's token
        Walk w = locate(S, B, Hkv, lo);
        int seg = 0, js = -w.t, je = w.n - w.t, ctx = ctx_s[w.b], draft0 = ctx - seq_of<kTok>(a, w.b, false).n;
        int t = (sl - js) * kTok + tok;
#pragma unroll 1
        for (int j = sl; j < cnt; j += 2, t += 2 * kTok) {
            if (j >= je) {
                while (j >= je) {
                    next_pair(w);
                    js = je;
                    je += w.n;
                    ++seg;
                }
                ctx = ctx_s[w.b];
                draft0 = ctx - seq_of<kTok>(a, w.b, false).n;
                t = (j - js) * kTok + tok;
            }
            landed();
            if (j >= 2 && !wait(KFREE0 + sl, ((j - 2) >> 1) & 1)) break;
            {
                const uint32_t src = ring + ru * L::kUnit + lane * RB + (sw << 4);   // chunk c: src ^ 16 c
                fence_after();
                constexpr int CH = RB / 16;
                uint4 x[CH];
#pragma unroll
                for (int c = 0; c < CH; ++c) x[c] = lds128(src ^ (c << 4));
#pragma unroll
                for (int q = 0; q < 4; ++q) {   // 32 channels at a time: 16 columns of fp16 pairs
                    uint32_t h[16];
                    if constexpr (I4) {
                        const uint32_t x4[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {   // channels in the order 0, 4, 1, 5, 2, 6, 3, 7
                            const uint32_t u = x4[k] ^ 0x88888888u, v = u >> 8;
                            h[4 * k] = nib_lo(u);
                            h[4 * k + 1] = nib_hi(u);
                            h[4 * k + 2] = nib_lo(v);
                            h[4 * k + 3] = nib_hi(v);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const uint4 y = x[(2 * q + c) % CH];
                            dec4<FMT>(y.x, h[8 * c], h[8 * c + 1]);
                            dec4<FMT>(y.y, h[8 * c + 2], h[8 * c + 3]);
                            dec4<FMT>(y.z, h[8 * c + 4], h[8 * c + 5]);
                            dec4<FMT>(y.w, h[8 * c + 6], h[8 * c + 7]);
                        }
                    }
                    tmem_st16(trow + sl * 64 + q * 16, reinterpret_cast<const float*>(h));
                }
                wait_st();
                fence_before();
                mbar_arrive(&bars[KFULL0 + sl]);
                read_done();
            }
            landed();
            uint32_t gs1[NG], gs2[NG];   // V's scales of this token x 2^2 (INT4) or 2^6 (INT8), as two fp16 terms, each twice
            if constexpr (NG > 1) {
                const uint4 raw = lds128(gring + gr * L::kGroups);
                if (++gr == L::kVUnits) gr = 0;
                const float g4[4] = {__uint_as_float(raw.x), __uint_as_float(raw.y), __uint_as_float(raw.z), __uint_as_float(raw.w)};
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    float s = t < ctx ? (ng == 4 ? g4[i] : g4[i / 2]) : 0.f;
                    // a draft token's scale that is not finite in fp16 must not reach the rows that do not see it
                    if (t >= draft0 && !(fabsf(s) < kMaxScale)) {
                        s = 0.f;
                        nan_seen[seg & (kSlots - 1)] = 1;
                    }
                    const float up = s * kScaleUp;
                    gs1[i] = pack_f16x2(up, up);
                    gs2[i] = residual(gs1[i], up, up);
                }
            }
            if (j >= 2 && !wait(VFREE0 + sl, ((j - 2) >> 1) & 1)) break;
            {
                const uint32_t src = ring + ru * L::kUnit + lane * RB + (sw << 4);   // chunk c: src ^ 16 c
                const uint32_t dst = sb + L::kV + sl * L::kVBuf + (tok >> 3) * 1024 + (tok & 7) * 144;   // (row, chunk tok % 8)
                // 8 fp16 codes of chunk ch (with group scales nib_lo4's or byte4_64's: stored as value and residual)
                auto put = [&](int ch, uint32_t h0, uint32_t h1, uint32_t h2, uint32_t h3) {
                    const uint32_t at = (dst ^ ((ch & 7) << 4)) + (ch >> 3) * kBlk;
                    if constexpr (NG == 1) {
                        sts128(at, h0, h1, h2, h3);
                    } else {
                        const uint32_t s1 = gs1[ch / 4 % NG], s2 = gs2[ch / 4 % NG];   // 32 channels per quarter of the row
                        const uint32_t h[4] = {h0, h1, h2, h3};
                        uint32_t hi[4], lw[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) scale_pair(h[i], s1, s2, hi[i], lw[i]);
                        sts128(at, hi[0], hi[1], hi[2], hi[3]);
                        sts128(at + kTileV, lw[0], lw[1], lw[2], lw[3]);
                    }
                };
                constexpr int CH = RB / 16;
                if (!kScaled && t >= draft0 && t < ctx) {
                    // a draft token's V: a code that is not finite must not reach the rows that do
                    // not see it.  Bit 7 of (code & 0x7F) + kUp says so for each byte of a word.
                    constexpr uint32_t kUp = FMT == E4M3 ? 0x01010101u : 0x04040404u;
                    auto bad = [](uint32_t u) { return ((u & 0x7F7F7F7Fu) + kUp) & 0x80808080u; };
#pragma unroll 2
                    for (int c = 0; c < CH; ++c) {
                        const uint4 y = lds128(src ^ (c << 4));
                        const uint4 m = make_uint4(bad(y.x), bad(y.y), bad(y.z), bad(y.w));
                        if (m.x | m.y | m.z | m.w) {
                            auto clean = [](uint32_t u, uint32_t w) { return u & ~((w >> 7) * 255u); };
                            sts128(src ^ (c << 4), clean(y.x, m.x), clean(y.y, m.y), clean(y.z, m.z), clean(y.w, m.w));
                            nan_seen[seg & (kSlots - 1)] = 1;
                        }
                    }
                }
                uint4 x[CH];
#pragma unroll
                for (int c = 0; c < CH; ++c) x[c] = lds128(src ^ (c << 4));
                if (t >= ctx) {   // past the context (INT4's zero code word is 0 too)
#pragma unroll
                    for (int c = 0; c < CH; ++c) x[c] = make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const uint32_t x4[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
                    if constexpr (I4) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t y = x4[k] ^ 0x88888888u, v = y >> 8;
                            if constexpr (NG == 1) put(4 * c + k, nib_lo(y), nib_hi(y), nib_lo(v), nib_hi(v));
                            else put(4 * c + k, nib_lo4(y), nib_hi4(y), nib_lo4(v), nib_hi4(v));
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint32_t h[4];
                            if constexpr (NG == 1) {
                                dec4<FMT>(x4[2 * k], h[0], h[1]);
                                dec4<FMT>(x4[2 * k + 1], h[2], h[3]);
                            } else {
                                byte4_64(x4[2 * k], h[0], h[1]);
                                byte4_64(x4[2 * k + 1], h[2], h[3]);
                            }
                            put(2 * c + k, h[0], h[1], h[2], h[3]);
                        }
                    }
                }
                fence_async();
                mbar_arrive(&bars[VFULL0 + sl]);
                read_done();
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
        // ---------------------------------------------------------- softmax ----
        const int g = warp >> 2, quad = warp & 3, tok = tid & 127;   // stream, lane quarter, token of the tile
        const uint32_t trow = tmem + ((uint32_t)(quad * 32) << 16);
        float* m_s = reinterpret_cast<float*>(sm + L::kM);
        float* mx_s = reinterpret_cast<float*>(sm + L::kMx) + g * 4 * RT;
        float* l_s = reinterpret_cast<float*>(sm + L::kL);
        float* f_s = reinterpret_cast<float*>(sm + L::kF);
        int* row_s = reinterpret_cast<int*>(sm + L::kRow);
        const float* mm = m_s + g * RT;   // the rows' maxima (less kUp): weights are 2^(z - mm)
        const float s_fp8 = (!kScaled && a.scale) ? __ldg(a.scale) : 1.0f;
        const float qk = a.sm_scale * s_fp8 * kLog2e;
        const int lbs = 31 - __clz(BS);
        float2* ws_ml = reinterpret_cast<float2*>(a.ws + verify_ml_off(plan.teams));
        float* ws_acc = reinterpret_cast<float*>(a.ws + verify_acc_off(plan.teams, RT));
        auto load16 = [](float (&y)[16], const float* p) {
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const float4 q = *reinterpret_cast<const float4*>(p + r);
                y[r] = q.x; y[r + 1] = q.y; y[r + 2] = q.z; y[r + 3] = q.w;
            }
        };
        Walk w = locate(S, B, Hkv, lo);
        int js = 0, segno = 0;
        while (js < cnt) {
            const Seq sq = seq_of<kTok>(a, w.b, false);
            const int P = sq.ctx - sq.n, R = min(RT, sq.n * G - cls * RT);
            const int seg = min(cnt - js, w.n - w.t);
            const int32_t* bt = a.block_tables + (int64_t)w.b * a.max_blocks_per_seq;
            // the rows of this row tile that see token t: G rows per query of the chunk that does
            auto rows_seeing = [&](int t) -> unsigned long long {
                if (t >= sq.ctx) return 0ull;
                if (t < P) return ~0ull;
                const int jt = t - P;
                unsigned long long rows = 0;
                const unsigned long long ones = G >= 64 ? ~0ull : (1ull << G) - 1ull;
#pragma unroll 4
                for (int i = 0; i < sq.n; ++i) {
                    const bool sees = a.tree_mask ? (__ldg(a.tree_mask + sq.q0 + i) >> jt) & 1ull : i >= jt;
                    const int at = i * G - cls * RT;   // the query's first row
                    if (sees && at < 64 && at > -64) rows |= at >= 0 ? ones << at : ones >> -at;
                }
                return rows;
            };
            if (tok < RT) m_s[g * RT + tok] = kNone;
            float l[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) l[r] = 0.f;
            bar_any(1 + g, 128, false);
            const int x0 = (js & 1) == g ? 0 : 1;   // this stream's first tile of the segment
            auto id_of = [&](int x) -> int {        // block of this thread's token in tile x of the segment
                const int t = (w.t + x) * kTok + tok;
                return kScaled && x < seg && t < sq.ctx ? __ldg(bt + (t >> lbs)) : -1;
            };
            // its scales: loaded one tile ahead, the block ids two
            float kn[NG], vn = 1.f;
            int id = id_of(x0);
            auto load_scales = [&]() {
#pragma unroll
                for (int i = 0; i < NG; ++i) kn[i] = kScaled ? 0.f : 1.f;
                vn = 1.f;
                if (kScaled && id >= 0 && id < a.cache.num_blocks) {
                    const int64_t row = ((int64_t)id * Hkv + w.kvh) * BS + (tok & (BS - 1));   // (BS divides kTok)
#pragma unroll
                    for (int i = 0; i < NG; ++i)
                        kn[i] = __ldg(a.cache.k_scales + row * (NG > 1 ? ng : 1) + ((i * ng) >> 2) * (NG > 1));
                    if (NG == 1) vn = __ldg(a.cache.v_scales + row);
                }
            };
            load_scales();
            id = id_of(x0 + 2);
#pragma unroll 1
            for (int x = x0; x < seg; x += 2) {
                const int j = js + x, t = (w.t + x) * kTok + tok;
                float k[NG], vs = vn;   // of this thread's token
                const float lv = kScaled && NG == 1 ? log2_scale(vs) : 0.f;   // (group scales are in V)
#pragma unroll
                for (int i = 0; i < NG; ++i) k[i] = qk * kn[i];
                if (kScaled) {
                    load_scales();
                    id = id_of(x + 4);
                }
                const int sx = j & (SB - 1);
                wait(SFULL0 + sx, (j >> kLogSB) & 1);
                fence_after();
                const uint32_t scol = trow + kColS + sx * NG * RT;
                // the groups' products with their scales, added up, of 16 rows
                auto logits = [&](float (&s)[16], int c0, auto less) {
                    [[maybe_unused]] float y[16];
                    tmem_ld16(scol + c0, s);
                    if constexpr (NG > 1) tmem_ld16(scol + RT + c0, y);
                    wait_ld();
                    reg_fence16(s);
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[r] = fmaf(s[r], k[0], -less(r));
                    if constexpr (NG > 1) {
#pragma unroll
                        for (int i = 1; i < NG; ++i) {
                            if (i > 1) {
                                tmem_ld16(scol + i * RT + c0, y);
                                wait_ld();
                            }
                            reg_fence16(y);
#pragma unroll
                            for (int r = 0; r < 16; ++r) s[r] = fmaf(y[r], k[i], s[r]);
                        }
                    }
                };
                const bool masked = (w.t + x + 1) * kTok > P;
                if (masked) {
                    // A tile that reaches into the chunk: its logits are masked in
                    // tensor memory (-inf where a row does not see the token), and
                    // the code below is the same for every tile.  A scale of V that
                    // is not finite becomes a NaN logit of the rows that see it.
                    const unsigned long long rows = rows_seeing(t);
                    const bool broken = kScaled && NG == 1 && !(fabsf(vs) < INFINITY);
                    if (broken) vs = 0.f;
#pragma unroll 1
                    for (int c0 = 0; c0 < RT; c0 += 16) {
                        float s[16];
                        logits(s, c0, [](int) { return 0.f; });
                        const uint32_t see = (uint32_t)(rows >> c0);
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            s[r] = (see >> r) & 1u ? (broken ? __int_as_float(0x7FC00000) : s[r]) : -INFINITY;
                        tmem_st16(scol + c0, s);
                        if constexpr (NG > 1) {
#pragma unroll
                            for (int r = 0; r < 16; ++r) s[r] = 0.f;
#pragma unroll
                            for (int i = 1; i < NG; ++i) tmem_st16(scol + i * RT + c0, s);
                        }
                    }
                    wait_st();
#pragma unroll
                    for (int i = 0; i < NG; ++i) k[i] = i == 0 ? 1.f : 0.f;
                }
                constexpr int kHeld = RT <= 32 ? RT / 16 : 1;   // 64 rows: read twice
                float top = -INFINITY, dd[kHeld][16];
#pragma unroll
                for (int c0 = 0; c0 < RT; c0 += 16) {
                    float(&s)[16] = dd[c0 / 16 % kHeld];
                    float q[16];
                    load16(q, mm + c0);
                    logits(s, c0, [&](int r) { return q[r]; });
#pragma unroll
                    for (int r = 0; r < 16; r += 2) top = fmax3(top, s[r], s[r + 1]);
                }
                bool held = RT <= 32;
                if (bar_any(1 + g, 128, top + lv > kLazy + kUp)) {
                    // New maxima over the tile's tokens, of the weights with V's scale.
                    held = false;
#pragma unroll 1
                    for (int c0 = 0; c0 < RT; c0 += 16) {
                        float v[16];
                        logits(v, c0, [&](int) { return kUp - lv; });
#pragma unroll
                        for (int r = 0; r < 16; ++r) v[r] = warp_max(v[r]);
                        if (lane == 0) {
                            float4* at = reinterpret_cast<float4*>(mx_s + quad * RT + c0);
#pragma unroll
                            for (int r = 0; r < 16; r += 4) at[r / 4] = make_float4(v[r], v[r + 1], v[r + 2], v[r + 3]);
                        }
                    }
                    bar_any(1 + g, 128, false);
                    if (tok < RT) {
                        // All rows, so that fewer tiles come here (E4M3, 32 x 8192 tokens: 101.7 us, 103.6 when only
                        // rows that exceed their own by 2^kLazy are raised); but in a tile that reaches into the chunk
                        // only those: what a row holds must not depend on tokens it does not see.
                        // (One that has seen nothing, or only NaN, keeps kNone.)
                        const float old = mm[tok];
                        const float tile = fmaxf(fmaxf(mx_s[tok], mx_s[RT + tok]), fmaxf(mx_s[2 * RT + tok], mx_s[3 * RT + tok]));
                        const float mn = tile > old + (masked ? kLazy : 0.f) ? tile : old;
                        f_s[g * RT + tok] = fast_exp2(old - mn);
                        m_s[g * RT + tok] = mn;
                    }
                    const bool o_live = x >= 2;   // O holds earlier tiles of the segment
                    if (o_live) {
                        wait(VFREE0 + g, ((j - 2) >> 1) & 1);
                        fence_after();
                    }
                    bar_any(1 + g, 128, false);
#pragma unroll
                    for (int c0 = 0; c0 < RT; c0 += 16) {
                        float al[16];
                        load16(al, f_s + g * RT + c0);
#pragma unroll
                        for (int r = 0; r < 16; ++r) l[c0 + r] *= al[r];
                    }
                    if (o_live) {
#pragma unroll 1
                        for (int c0 = 0; c0 < 2 * RT; c0 += 16) {   // both halves' columns
                            float o[16], al[16];
                            const uint32_t col = trow + kColO + g * 2 * RT + c0;
                            tmem_ld16(col, o);
                            load16(al, f_s + g * RT + (c0 & (RT - 1)));
                            wait_ld();
                            reg_fence16(o);
#pragma unroll
                            for (int r = 0; r < 16; ++r) o[r] *= al[r];
                            tmem_st16(col, o);
                        }
                        wait_st();
                    }
                }
                if (held) {   // S is in registers
                    fence_before();
                    mbar_arrive(&bars[SFREE0 + sx]);
                }
                if (j >= 2) wait(VFREE0 + g, ((j - 2) >> 1) & 1);   // P's buffer is free
                const uint32_t prow = sb + L::kP + g * L::kPBlocks * kBlk + (tok >> 3) * 1024 + (tok & 7) * 128;
#pragma unroll
                for (int c0 = 0; c0 < RT; c0 += 16) {
                    float(&s)[16] = dd[c0 / 16 % kHeld];
                    if (!held) {
                        float q[16];
                        load16(q, mm + c0);
                        logits(s, c0, [&](int r) { return q[r]; });
                    }
                    uint32_t hi[8], lw[8];
#pragma unroll
                    for (int r = 0; r < 16; r += 2) {
                        float p0 = fast_exp2(s[r]), p1 = fast_exp2(s[r + 1]);
                        l[c0 + r] += p0;
                        l[c0 + r + 1] += p1;
                        if (kScaled && NG == 1) {   // (group scales are in V)
                            p0 *= vs;
                            p1 *= vs;
                        }
                        hi[r / 2] = pack_f16x2(p0, p1);
                        lw[r / 2] = residual(hi[r / 2], p0, p1);
                    }
                    // columns c0 .. of P_hi, RT + c0 .. of P_lo
#pragma unroll
                    for (int hl = 0; hl < 2; ++hl)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const uint32_t ch = (hl * RT + c0) / 8 + q;
                            const uint32_t* h = hl ? lw : hi;
                            sts128(prow + (ch >> 3) * kBlk + (((ch & 7) ^ (tok & 7)) << 4), h[4 * q], h[4 * q + 1], h[4 * q + 2], h[4 * q + 3]);
                        }
                }
                fence_async();
                fence_before();
                if (!held) mbar_arrive(&bars[SFREE0 + sx]);
                mbar_arrive(&bars[PFULL0 + g]);
            }
            // ------------------------------------------------- segment end ----
            const int last = x0 < seg ? x0 + (seg - 1 - x0) / 2 * 2 : -1;   // this stream's last tile
            // sums over the warp's 32 tokens: 16 rows at a time, lane r ends with row r's
#pragma unroll
            for (int c0 = 0; c0 < RT; c0 += 16) {
#pragma unroll
                for (int wd = 8; wd >= 1; wd >>= 1) {
#pragma unroll
                    for (int r = 0; r < wd; ++r) {
                        const bool up = lane & wd;
                        const float give = up ? l[c0 + r] : l[c0 + r + wd], own = up ? l[c0 + r + wd] : l[c0 + r];
                        l[c0 + r] = own + __shfl_xor_sync(0xFFFFFFFFu, give, wd);
                    }
                }
                l[c0] += __shfl_xor_sync(0xFFFFFFFFu, l[c0], 16);
                if (lane < 16) l_s[(g * 4 + quad) * RT + c0 + lane] = l[c0];
            }
            asm volatile("bar.sync 3, 256;" ::: "memory");   // both streams' maxima and sums
            const bool whole = seg == w.n;
            const int slot = blockIdx.x * 2 + (w.t == 0 ? 1 : 0);
            if (tid < RT) {   // a row's factors of the two streams (a stream without a tile: 0)
                const float m0 = m_s[tid], m1 = m_s[RT + tid], M = fmaxf(m0, m1);
                const bool h0 = seg > 1 || (js & 1) == 0, h1 = seg > 1 || (js & 1) == 1;
                float f0 = h0 ? fast_exp2(m0 - M) : 0.f, f1 = h1 ? fast_exp2(m1 - M) : 0.f;
                const float* q = l_s + tid;
                const float sum = ((q[0] + q[RT]) + (q[2 * RT] + q[3 * RT])) * f0 + ((q[4 * RT] + q[5 * RT]) + (q[6 * RT] + q[7 * RT])) * f1;
                if (!whole && tid < R) ws_ml[(int64_t)slot * RT + tid] = make_float2(M, sum);
                const float inv = whole ? (sum == 0.f ? 0.f : s_fp8 / sum) : s_fp8;
                f_s[tid] = f0 * inv;
                f_s[RT + tid] = f1 * inv;
                const int qr = cls * RT + tid;
                row_s[tid] = qr / G * a.num_q_heads + w.kvh * G + qr % G;
            }
            if (last >= 0) wait(VFREE0 + g, ((js + last) >> 1) & 1);
            asm volatile("bar.sync 3, 256;" ::: "memory");   // both streams' products, the factors
            fence_after();
            unsigned long long nan_rows = 0;   // rows whose channel is NaN
            const int ch = quad * 32 + lane;   // this thread's row of O^T
            const int d = I4 ? (ch & ~7) | ((ch & 1) << 2) | ((ch & 7) >> 1) : ch;   // its channel
            if ((!kScaled || NG > 1) && nan_seen[segno & (kSlots - 1)]) {
                for (int t = max(P, w.t * kTok); t < min(sq.ctx, (w.t + seg) * kTok); ++t) {
                    const int bid = __ldg(bt + (t >> lbs));
                    if (bid < 0 || bid >= a.cache.num_blocks) continue;
                    const int64_t row = ((int64_t)bid * Hkv + w.kvh) * BS + (t & (BS - 1));
                    bool bad;
                    if constexpr (NG > 1) {
                        bad = !(fabsf(a.cache.v_scales[row * ng + d * ng / D]) < kMaxScale);
                    } else {
                        const int c = a.cache.v_codes[row * RB + d] & 0x7F;
                        bad = FMT == E4M3 ? c == 0x7F : c > 0x7B;
                    }
                    if (bad) nan_rows |= rows_seeing(t);
                }
            }
            constexpr int HR = RT / 2, N = HR < 16 ? HR : 16;   // rows of each stream's threads
            uint16_t* const od = a.out + (int64_t)sq.q0 * a.num_q_heads * D + d;
            float* const pd = ws_acc + (int64_t)slot * RT * D + d;
#pragma unroll 1
            for (int r0 = g * HR; r0 < g * HR + HR; r0 += 16) {
                const int rb = RT == 16 ? 0 : r0;   // (tiles of 16: both streams' threads add up all of them)
                float o[16], y[2][16], z[2][16];   // values and residuals' columns of both streams
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    const uint32_t col = trow + kColO + st * 2 * RT + rb;
                    tmem_ld16(col, y[st]);
                    tmem_ld16(col + RT, z[st]);
                }
                wait_ld();
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    reg_fence16(y[st]);
                    reg_fence16(z[st]);
                    float f[16];
                    load16(f, f_s + st * RT + rb);
                    const bool written = seg > 1 || st == (js & 1);
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const float v = written ? (y[st][r] + z[st][r]) * f[r] : 0.f;
                        o[r] = st == 0 ? v : o[r] + v;
                    }
                }
                if (RT == 16 && g) {
#pragma unroll
                    for (int r = 0; r < N; ++r) o[r] = o[(r + N) & 15];
                }
                if (nan_rows) {
#pragma unroll
                    for (int r = 0; r < N; ++r)
                        if ((nan_rows >> (r0 + r)) & 1ull) o[r] = __int_as_float(0x7FC00000);
                }
                if (whole) {
#pragma unroll
                    for (int r = 0; r < N; r += 4) {
                        const int4 at = *reinterpret_cast<const int4*>(row_s + r0 + r);
                        const int at4[4] = {at.x, at.y, at.z, at.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (r0 + r + k < R) od[(int64_t)at4[k] * D] = __half_as_ushort(__float2half_rn(o[r + k]));
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < N; ++r)
                        if (r0 + r < R) pd[(r0 + r) * D] = o[r];
                }
            }
            fence_before();
            asm volatile("bar.sync 3, 256;" ::: "memory");   // maxima, sums and factors read by everyone
            if (tid == 0) {
                nan_seen[segno & (kSlots - 1)] = 0;
                if (js + seg == cnt) {   // the last segment: parts of it that later CTAs hold
                    *hdr = make_int4(w.b, w.kvh, cls, w.t == 0 ? sh.parts : 0);
                }
            }
            mbar_arrive(&bars[OFREE]);
            js += seg;
            ++segno;
            if (js < cnt) next_pair(w);
        }
        fence_before();
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        if (cnt > 0 && lane == 0) mbar_wait(&bars[OFINAL], 0, nullptr);   // every issued MMA has completed
        __syncwarp();
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
    }
}

template <int FMT, int RT, int NG>
cudaError_t launch_t(const VerifyArgs& a, const VerifyPlan& p, cudaStream_t s) {
    auto kern = verify_tc_kernel<FMT, RT, NG>;
    const int smem = (int)Smem<FMT, RT, NG>::bytes(a.batch);
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = once_per_device(done, [&]() -> cudaError_t {
        // the warpgroups' register split draws on what the launch holds
        cudaFuncAttributes f;
        cudaError_t r = cudaFuncGetAttributes(&f, kern);
        if (r != cudaSuccess) return r;
        if (f.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Smem<FMT, RT, NG>::bytes(kMaxBatch));
    });
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3((unsigned)p.ctas), dim3(kThreads), smem, s, a, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(verify_reduce_kernel<D>, dim3((unsigned)p.teams, (unsigned)(RT / 8)), dim3(256), 0, s, a, p);
}

template <int FMT>
cudaError_t launch_fmt(const VerifyArgs& a, const VerifyPlan& p, cudaStream_t s) {
    if constexpr (FMT == INT8 || FMT == INT4) {
        if (a.cache.ngroups > 1) return p.rows == 16 ? launch_t<FMT, 16, 4>(a, p, s) : launch_t<FMT, 32, 4>(a, p, s);
    }
    if (p.rows == 16) return launch_t<FMT, 16, 1>(a, p, s);
    if (p.rows == 32) return launch_t<FMT, 32, 1>(a, p, s);
    return launch_t<FMT, 64, 1>(a, p, s);
}

}  // namespace tc
}  // namespace verify
}  // namespace kvq
