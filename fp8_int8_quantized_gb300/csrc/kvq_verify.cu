// How a chunk-attention call is cut up, and the choice of its format's kernels.
#include <algorithm>

#include "kvq_verify.cuh"

namespace kvq {

VerifyPlan plan_verify(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t ngroups,
                       int32_t max_query_len, int32_t max_context_len, int32_t sms) {
    VerifyPlan p;
    const int rows = max_query_len * (num_q_heads / num_kv_heads);
    // tcgen05 for every head_dim-128 call whose batch fits its shared memory; measured
    // against the mma.sync kernels (us, L2 flushed before each call, tcgen05 / mma.sync):
    //   E4M3, 32 x 8192 tokens, 8 kv-heads: 1 row 111 / 127, 8 rows 112 / 129, 32 rows 117 / 225
    //   E5M2, ragged trees of 36 .. 64 rows: 88 / 199; one sequence of 1000, 16 rows: 17 / 17
    //   INT8, 16 x 4096, 40 kv-heads: 1 row 135 / 158, 8 rows 137 / 160
    //   INT4, 32-channel groups, 3 x ~115000, 40 .. 56 rows: 356 / 775
    p.tc = head_dim == 128 && batch <= kMaxTcBatch;
    const int tile = p.tc ? 128 : verify::kTile;
    // 64 rows per row tile where tensor memory holds their logits (not one product per scale
    // group): V and K are converted once instead of twice
    p.rows = p.tc ? (rows <= 16 ? 16 : rows <= 32 || ngroups > 1 ? 32 : 64) : (rows <= 8 ? 8 : rows <= 16 ? 16 : 32);
    p.row_tiles = (rows + p.rows - 1) / p.rows;
    const int64_t tiles = (int64_t)batch * num_kv_heads * p.row_tiles * (((int64_t)max_context_len + tile - 1) / tile);
    if (p.tc) {
        p.warps = p.team = 1;
        p.ctas = (int32_t)std::max<int64_t>(std::min<int64_t>(sms, tiles), std::min(p.row_tiles, sms));
        p.teams = p.ctas;
        return p;
    }
    p.warps = 8;
    // A partial result is `rows` x head_dim fp32 values; with a range per warp every warp may leave
    // two, with a range per CTA every (sequence, kv-head) it meets ends in a merge of its 8 warps.
    // Range per warp / per CTA, us, head_dim 64, 8 kv-heads, E4M3, 8 or 2 rows (tiles per warp):
    //   8 sequences of 2432 (4)    21.2 / 18.0     8 x 4864 (8)   26.7 / 22.8     8 x 7296 (12)  32.1 / 29.0
    //   128 x 333 .. 1000 (27)     40.5 / 62.6     64 x 1333 .. 4000 (53) 63.7 / 74.9
    //   1024 x 83 .. 250 (54)      89.8 / 197      4096 x 20 .. 60 (54)   181 / 704
    // so 12 tiles per warp part the two where a batch is large; with fewer pairs than CTAs a range per CTA
    // stays 5 to 10% ahead beyond them (8 x 29184, 48 tiles per warp: 81.5 / 77.6).
    p.team = tiles >= (int64_t)sms * p.warps * 12 ? 1 : p.warps;
    const int64_t want = p.team == 1 ? sms : (tiles + p.warps - 1) / p.warps;
    p.ctas = (int32_t)std::max<int64_t>(std::min<int64_t>(sms, want), std::min(p.row_tiles, sms));
    p.teams = p.team == 1 ? p.ctas * p.warps : p.ctas;
    return p;
}

cudaError_t launch_verify(const VerifyArgs& a, const VerifyPlan& p, cudaStream_t s) {
    switch (a.cache.fmt) {
        case E4M3: return verify::launch_e4m3(a, p, s);
        case E5M2: return verify::launch_e5m2(a, p, s);
        case INT4: return verify::launch_int4(a, p, s);
        default: return verify::launch_int8(a, p, s);
    }
}

}  // namespace kvq
