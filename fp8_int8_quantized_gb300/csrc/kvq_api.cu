// C ABI of the kvq library: argument validation, status codes, workspace
// sizing, context-split choice and the per-device error word.  Every entry
// point validates before it launches anything, so a call that returns an
// error has written nothing.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "../../include/kvq.h"
#include "kvq_device.cuh"
#include "kvq_launch.h"
#include "kvq_spec.h"

namespace kvq {
// The debug FP8 encoder's launcher (kvq_dequant.cu).
cudaError_t launch_encode_fp8(const float* x, uint8_t* codes, int64_t n, int fmt, cudaStream_t s);
}  // namespace kvq

namespace {

// First error a kernel met on this device: code << 56 | detail.
__device__ unsigned long long g_kvq_err = 0;

constexpr int kMaxDevices = 64;
std::mutex g_mu;
unsigned long long* g_err_ptr[kMaxDevices] = {};
int g_sm_count[kMaxDevices] = {};
std::atomic<int> g_decode_kernel{0};
cudaEvent_t g_ev_begin = nullptr, g_ev_end = nullptr;

constexpr int kMaxChunkTokens = 65536;
constexpr int kMaxBatch = 4096;   // the decode kernel scans the context lengths in shared memory

bool current_device(int* dev) {
    if (cudaGetDevice(dev) != cudaSuccess) return false;
    return *dev >= 0 && *dev < kMaxDevices;
}

unsigned long long* err_word(int dev) {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_err_ptr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_kvq_err) != cudaSuccess) return nullptr;
        g_err_ptr[dev] = static_cast<unsigned long long*>(p);
    }
    return g_err_ptr[dev];
}

int sm_count(int dev) {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_sm_count[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
        g_sm_count[dev] = n;
    }
    return g_sm_count[dev];
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Whether two sets of n rows of 16-bit elements (x_row elements, x_stride >= x_row apart, from x on; y
// likewise) share any.  Rows of one buffer side by side, such as a fused QKV buffer's, do not.
bool rows_overlap(const void* x, int64_t x_stride, int64_t x_row, const void* y, int64_t y_stride, int64_t y_row, int64_t n) {
    const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(y) - reinterpret_cast<uintptr_t>(x)) / 2;
    if (d >= (n - 1) * x_stride + x_row || -d >= (n - 1) * y_stride + y_row) return false;
    const auto floor_div = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };
    if (x_stride == y_stride) {   // row t of y starts at element r of x's place t + j
        const int64_t j = floor_div(d, x_stride), r = d - j * x_stride;
        return (r < x_row && j < n && -j < n) || (r + y_row > x_stride && j + 1 < n && -(j + 1) < n);
    }
    for (int64_t t = 0; t < n; ++t) {   // the last row of x that starts before the end of y's row t
        const int64_t a = d + t * y_stride, u = std::min(n - 1, floor_div(a + y_row - 1, x_stride));
        if (u >= 0 && u * x_stride + x_row > a) return true;
    }
    return false;
}

kvq_status check_cache(const kvq_cache* c, int32_t fmt) {
    if (!c) return KVQ_ERR_INVALID_ARG;
    if (fmt != KVQ_E4M3 && fmt != KVQ_E5M2 && fmt != KVQ_INT8 && fmt != KVQ_INT4) return KVQ_ERR_INVALID_ARG;
    if (c->fmt != fmt) return KVQ_ERR_INVALID_ARG;
    if (!c->k_codes || !c->v_codes || !aligned(c->k_codes, 16) || !aligned(c->v_codes, 16))
        return KVQ_ERR_INVALID_ARG;
    if (c->num_blocks <= 0 || c->num_kv_heads <= 0) return KVQ_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return KVQ_ERR_UNSUPPORTED;
    if (c->block_size != 16 && c->block_size != 32 && c->block_size != 64) return KVQ_ERR_UNSUPPORTED;
    if (fmt == KVQ_INT8 || fmt == KVQ_INT4) {
        if (!c->k_scales || !c->v_scales || !aligned(c->k_scales, 16) || !aligned(c->v_scales, 16))
            return KVQ_ERR_INVALID_ARG;
        const int32_t g = c->group_size;
        if (g != 0 && g != c->head_dim && g != c->head_dim / 2 && g != c->head_dim / 4) return KVQ_ERR_INVALID_ARG;
    } else if (c->group_size != 0) {
        return KVQ_ERR_INVALID_ARG;
    }
    // TMA row coordinates are 32-bit
    if ((int64_t)c->num_blocks * c->num_kv_heads * c->block_size > 0x7FFFFFFFll) return KVQ_ERR_UNSUPPORTED;
    return KVQ_OK;
}

kvq::CacheView view(const kvq_cache* c) {
    const int32_t ng = c->group_size > 0 ? c->head_dim / c->group_size : 1;
    return kvq::CacheView{static_cast<uint8_t*>(c->k_codes), static_cast<uint8_t*>(c->v_codes), c->k_scales,
                          c->v_scales, c->num_blocks, c->block_size, c->num_kv_heads, c->head_dim, c->fmt, ng};
}

// Decode tiles (kDecodeTileTokens tokens) per context chunk.  Every warp of the persistent decode
// kernel streams a contiguous range of the flat tile list that is at least one
// chunk long; chunks of about half a range keep every warp busy while the
// partial slots stay few (two per chunk).  Counts 16 warps per SM (the kernel
// runs 12, and 16 for INT4), so chunks come out at 0.4-0.5 of a range.
int32_t choose_chunk_tiles(int32_t batch, int32_t num_kv_heads, int32_t group, int32_t max_ctx, int sms) {
    constexpr int TT = kvq::kDecodeTileTokens;
    const int64_t tiles = (int64_t)batch * num_kv_heads * ((max_ctx + TT - 1) / TT);
    const int64_t warps = (int64_t)sms * 16;
    int64_t c = tiles / (2 * warps);
    // Small batches: short chunks spread the few tiles over many warps; the
    // partial slots a chunk writes (G q-heads x head_dim + 2 floats, twice)
    // stay below ~1/8 of its cache bytes with at least G / 2 tiles per chunk,
    // and one-tile chunks cost more in flushes than they gain (Llama-2-7B
    // shapes at batch 4: 31 us per step against 27 with two-tile chunks).
    const int64_t cmin = group > 4 ? group / 2 : 2;
    if (c < cmin) c = cmin;
    if (c > 256) c = 256;
    return (int32_t)c;
}

int32_t resolve_chunk_tiles(int32_t partition_size, int32_t batch, int32_t num_kv_heads, int32_t group,
                            int32_t max_ctx) {
    if (partition_size > 0) return partition_size / kvq::kDecodeTileTokens;
    int dev = 0;
    if (!current_device(&dev)) dev = 0;
    return choose_chunk_tiles(batch, num_kv_heads, group, max_ctx, sm_count(dev));
}

kvq_status decode_impl(const void* q, const void* k_new, const void* v_new, const kvq_cache* cache,
                       const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
                       int32_t batch, int32_t num_q_heads, int32_t max_context_len, const float* scale, int32_t fmt,
                       float sm_scale, void* out, void* workspace, size_t workspace_bytes, int32_t partition_size,
                       kvq_stream_t stream) {
    kvq_status st = check_cache(cache, fmt);
    if (st != KVQ_OK) return st;
    if (batch < 0 || num_q_heads <= 0 || max_context_len < 0 || max_blocks_per_seq <= 0) return KVQ_ERR_INVALID_ARG;
    if (num_q_heads % cache->num_kv_heads) return KVQ_ERR_INVALID_ARG;
    const int G = num_q_heads / cache->num_kv_heads;
    if (G > 8) return KVQ_ERR_UNSUPPORTED;
    // (the tensor-core consumer carries one operand row per (q-head, scale
    // group), eight per launch: more take several launches over the same tiles)
    if ((int64_t)max_blocks_per_seq * cache->block_size < max_context_len) return KVQ_ERR_INVALID_ARG;
    if (batch > 65535 || cache->num_kv_heads > 65535 || num_q_heads > 65535) return KVQ_ERR_UNSUPPORTED;
    if (batch == 0) return KVQ_OK;
    if (!q || !block_tables || !context_lens || !out || !aligned(q, 16) || !aligned(out, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4))
        return KVQ_ERR_INVALID_ARG;
    if (scale && !aligned(scale, 4)) return KVQ_ERR_INVALID_ARG;
    if (!(sm_scale >= 0.f) || std::isinf(sm_scale)) return KVQ_ERR_INVALID_ARG;
    if (partition_size < 0 || partition_size % 64 || partition_size > kMaxChunkTokens) return KVQ_ERR_INVALID_ARG;
    if (batch > kMaxBatch) return KVQ_ERR_UNSUPPORTED;
    constexpr int TT = kvq::kDecodeTileTokens;
    if ((int64_t)batch * cache->num_kv_heads * ((max_context_len + TT - 1) / TT) >= 0x7FFFFFFFll)
        return KVQ_ERR_UNSUPPORTED;  // flat tile indices are 32-bit
    const int32_t C = resolve_chunk_tiles(partition_size, batch, cache->num_kv_heads, G, max_context_len);
    const int32_t nch = std::max<int32_t>(1, ((max_context_len + TT - 1) / TT + C - 1) / C);
    const size_t need = kvq::ws_bytes(batch, num_q_heads, nch, cache->head_dim);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return KVQ_ERR_WORKSPACE;
    int kind = g_decode_kernel.load();
    if (kind == 0) kind = 2;
    // CUDA-core kernel: 8-bit codes, G <= 4
    if (kind == 1 && (G > 4 || fmt == KVQ_INT4)) return KVQ_ERR_UNSUPPORTED;
    int dev;
    if (!current_device(&dev)) return KVQ_ERR_CUDA;
    unsigned long long* err = err_word(dev);
    if (!err) return KVQ_ERR_CUDA;
    kvq::DecodeArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.cache = view(cache);
    a.block_tables = block_tables;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.context_lens = context_lens;
    a.batch = batch;
    a.num_q_heads = num_q_heads;
    a.max_context_len = max_context_len;
    a.scale = (fmt == KVQ_INT8 || fmt == KVQ_INT4) ? nullptr : scale;
    a.sm_scale = sm_scale > 0.f ? sm_scale : 1.0f / std::sqrt((float)cache->head_dim);
    a.out = static_cast<uint16_t*>(out);
    a.ws = static_cast<float*>(workspace);
    a.chunk_tiles = C;
    a.num_chunks = nch;
    a.kernel = kind;
    a.err = err;
    a.ev_begin = g_ev_begin;
    a.ev_end = g_ev_end;
    a.k_new = static_cast<const uint16_t*>(k_new);
    a.v_new = static_cast<const uint16_t*>(v_new);
    return kvq::launch_decode(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace

extern "C" {

int32_t kvq_abi_version(void) { return KVQ_ABI_VERSION; }

const char* kvq_status_string(kvq_status s) {
    switch (s) {
        case KVQ_OK: return "ok";
        case KVQ_ERR_INVALID_ARG: return "invalid argument";
        case KVQ_ERR_UNSUPPORTED: return "unsupported size (head_dim, block_size or group size)";
        case KVQ_ERR_WORKSPACE: return "workspace missing or too small";
        case KVQ_ERR_OUT_OF_RANGE: return "a slot, block id or context length was outside the cache";
        case KVQ_ERR_TIMEOUT: return "a kernel's bounded wait ran out";
        case KVQ_ERR_CUDA: return "CUDA runtime error";
        case KVQ_ERR_SCRATCH_LIMIT: return "needs more scratch than the library's fixed device array";
    }
    return "unknown status";
}

void kvq_set_decode_timing_events(void* ev_begin, void* ev_end) {
    if (ev_begin && ev_end) {
        g_ev_begin = static_cast<cudaEvent_t>(ev_begin);
        g_ev_end = static_cast<cudaEvent_t>(ev_end);
    } else {
        g_ev_begin = g_ev_end = nullptr;
    }
}

int32_t kvq_set_decode_kernel(int32_t kind) {
    if (kind < 0 || kind > 2) return -1;
    return g_decode_kernel.exchange(kind);
}

kvq_status kvq_append(const void* k, const void* v, const kvq_cache* cache, const int64_t* slot_mapping,
                      int64_t num_tokens, const float* scale, int32_t fmt, kvq_stream_t stream) {
    kvq_status st = check_cache(cache, fmt);
    if (st != KVQ_OK) return st;
    if (num_tokens < 0) return KVQ_ERR_INVALID_ARG;
    if (num_tokens == 0) return KVQ_OK;
    if (!k || !v || !slot_mapping || !aligned(k, 16) || !aligned(v, 16) || !aligned(slot_mapping, 8))
        return KVQ_ERR_INVALID_ARG;
    if (scale && !aligned(scale, 4)) return KVQ_ERR_INVALID_ARG;
    if (num_tokens * cache->num_kv_heads * (cache->head_dim / 16) / 256 >= 0x7FFFFFFFll) return KVQ_ERR_UNSUPPORTED;
    int dev;
    if (!current_device(&dev)) return KVQ_ERR_CUDA;
    unsigned long long* err = err_word(dev);
    if (!err) return KVQ_ERR_CUDA;
    kvq::AppendArgs a{static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), view(cache), slot_mapping,
                      num_tokens, (fmt == KVQ_INT8 || fmt == KVQ_INT4) ? nullptr : scale, err};
    return kvq::launch_append(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

size_t kvq_decode_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                 int32_t max_context_len, int32_t partition_size) {
    if (batch <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || max_context_len < 0) return 0;
    if (num_q_heads % num_kv_heads) return 0;
    const int32_t C = resolve_chunk_tiles(partition_size, batch, num_kv_heads, num_q_heads / num_kv_heads,
                                          max_context_len);
    if (C <= 0) return 0;
    constexpr int TT = kvq::kDecodeTileTokens;
    const int64_t nch = std::max<int64_t>(1, ((max_context_len + TT - 1) / TT + C - 1) / C);
    return kvq::ws_bytes(batch, num_q_heads, nch, head_dim);
}

kvq_status kvq_decode_attention(const void* q, const kvq_cache* cache, const int32_t* block_tables,
                                int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t batch,
                                int32_t num_q_heads, int32_t max_context_len, const float* scale, int32_t fmt,
                                float sm_scale, void* out, void* workspace, size_t workspace_bytes,
                                int32_t partition_size, kvq_stream_t stream) {
    return decode_impl(q, nullptr, nullptr, cache, block_tables, max_blocks_per_seq, context_lens, batch,
                       num_q_heads, max_context_len, scale, fmt, sm_scale, out, workspace, workspace_bytes,
                       partition_size, stream);
}

kvq_status kvq_decode_attention_append(const void* q, const void* k_new, const void* v_new, const kvq_cache* cache,
                                       const int32_t* block_tables, int32_t max_blocks_per_seq,
                                       const int32_t* context_lens, int32_t batch, int32_t num_q_heads,
                                       int32_t max_context_len, const float* scale, int32_t fmt, float sm_scale,
                                       void* out, void* workspace, size_t workspace_bytes, int32_t partition_size,
                                       kvq_stream_t stream) {
    if (batch > 0 && (!k_new || !v_new || !aligned(k_new, 16) || !aligned(v_new, 16))) return KVQ_ERR_INVALID_ARG;
    return decode_impl(q, k_new, v_new, cache, block_tables, max_blocks_per_seq, context_lens, batch, num_q_heads,
                       max_context_len, scale, fmt, sm_scale, out, workspace, workspace_bytes, partition_size,
                       stream);
}

kvq_status kvq_prefill_attention(const void* q, const kvq_cache* cache, const int32_t* block_tables,
                                 int32_t max_blocks_per_seq, const int32_t* context_lens, const int32_t* query_start,
                                 int32_t batch, int64_t num_q_tokens, int32_t num_q_heads, int32_t max_query_len,
                                 const float* scale,
                                 int32_t fmt, float sm_scale, void* out, kvq_stream_t stream) {
    kvq_status st = check_cache(cache, fmt);
    if (st != KVQ_OK) return st;
    if (batch < 0 || num_q_tokens < 0 || num_q_heads <= 0 || max_query_len < 0 || max_blocks_per_seq <= 0)
        return KVQ_ERR_INVALID_ARG;
    if (num_q_heads % cache->num_kv_heads) return KVQ_ERR_INVALID_ARG;
    if (num_q_heads / cache->num_kv_heads > kvq::prefill_rows_per_tile()) return KVQ_ERR_UNSUPPORTED;
    if (num_q_tokens > 0x7FFFFFFFll) return KVQ_ERR_UNSUPPORTED;   // query_start entries are int32
    if (batch > 65535 || cache->num_kv_heads > 65535) return KVQ_ERR_UNSUPPORTED;
    if (batch == 0 || max_query_len == 0 || num_q_tokens == 0) return KVQ_OK;
    if (!q || !block_tables || !context_lens || !query_start || !out || !aligned(q, 16) || !aligned(out, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(query_start, 4))
        return KVQ_ERR_INVALID_ARG;
    if (scale && !aligned(scale, 4)) return KVQ_ERR_INVALID_ARG;
    if (!(sm_scale >= 0.f) || std::isinf(sm_scale)) return KVQ_ERR_INVALID_ARG;
    int dev;
    if (!current_device(&dev)) return KVQ_ERR_CUDA;
    unsigned long long* err = err_word(dev);
    if (!err) return KVQ_ERR_CUDA;
    kvq::PrefillArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.cache = view(cache);
    a.block_tables = block_tables;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.batch = batch;
    a.num_q_tokens = num_q_tokens;
    a.num_q_heads = num_q_heads;
    a.max_query_len = max_query_len;
    a.scale = (fmt == KVQ_INT8 || fmt == KVQ_INT4) ? nullptr : scale;
    a.sm_scale = sm_scale > 0.f ? sm_scale : 1.0f / std::sqrt((float)cache->head_dim);
    a.out = static_cast<uint16_t*>(out);
    a.err = err;
    return kvq::launch_prefill(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_append_rotary(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                             int64_t v_stride, int32_t dtype, int32_t num_q_heads, const kvq_cache* cache,
                             const int64_t* slot_mapping, int64_t num_tokens, const int64_t* positions,
                             int32_t num_axes, const uint8_t* axis_of_pair, const float* cos_sin,
                             int64_t max_position, int32_t rot_dim, int32_t interleaved, const float* scale,
                             int32_t fmt, void* q_out, int64_t q_out_stride, kvq_stream_t stream) {
    kvq_status st = check_cache(cache, fmt);
    if (st != KVQ_OK) return st;
    if (num_tokens < 0 || num_q_heads < 0 || (dtype != KVQ_F16 && dtype != KVQ_BF16)) return KVQ_ERR_INVALID_ARG;
    const int64_t D = cache->head_dim, Hkv = cache->num_kv_heads;
    if (rot_dim <= 0 || rot_dim > D || rot_dim % 2 || max_position <= 0) return KVQ_ERR_INVALID_ARG;
    if (rot_dim % 16) return KVQ_ERR_UNSUPPORTED;
    if (num_axes < 1 || (num_axes > 1 && !axis_of_pair)) return KVQ_ERR_INVALID_ARG;
    if (num_axes > KVQ_MAX_AXES) return KVQ_ERR_UNSUPPORTED;
    if (num_tokens == 0) return KVQ_OK;
    // the launch's warps: at most one per four head rows of a token
    if (num_tokens > (int64_t)1 << 31 || num_tokens * ((num_q_heads + 3) / 4 + 2 * ((Hkv + 3) / 4)) / 4 >= 0x7FFFFFFFll)
        return KVQ_ERR_UNSUPPORTED;
    if (!k || !v || !slot_mapping || !positions || !cos_sin || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(slot_mapping, 8) || !aligned(positions, 8) || !aligned(cos_sin, 16) || !aligned(axis_of_pair, 8))
        return KVQ_ERR_INVALID_ARG;
    if (scale && !aligned(scale, 4)) return KVQ_ERR_INVALID_ARG;
    if (k_stride % 8 || v_stride % 8 || k_stride < Hkv * D || v_stride < Hkv * D) return KVQ_ERR_INVALID_ARG;
    if (num_q_heads > 0) {
        if (!q || !q_out || !aligned(q, 16) || !aligned(q_out, 16)) return KVQ_ERR_INVALID_ARG;
        const int64_t row = num_q_heads * D;
        if (q_stride % 8 || q_out_stride % 8 || q_stride < row || q_out_stride < row) return KVQ_ERR_INVALID_ARG;
        // in place (the same fp16 rows) or apart; K and V are read while q_out is written
        const bool same = q == q_out && (q_stride == q_out_stride || num_tokens == 1) && dtype == KVQ_F16;
        if ((!same && rows_overlap(q, q_stride, row, q_out, q_out_stride, row, num_tokens)) ||
            rows_overlap(k, k_stride, Hkv * D, q_out, q_out_stride, row, num_tokens) ||
            rows_overlap(v, v_stride, Hkv * D, q_out, q_out_stride, row, num_tokens))
            return KVQ_ERR_INVALID_ARG;
    }
    int dev;
    if (!current_device(&dev)) return KVQ_ERR_CUDA;
    unsigned long long* err = err_word(dev);
    if (!err) return KVQ_ERR_CUDA;
    kvq::RotaryArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out = static_cast<uint16_t*>(q_out);
    a.qo_stride = q_out_stride;
    a.cache = view(cache);
    a.slot_mapping = slot_mapping;
    a.positions = positions;
    a.axis_of_pair = axis_of_pair;
    a.cos_sin = cos_sin;
    a.max_position = max_position;
    a.num_tokens = num_tokens;
    a.num_axes = num_axes;
    a.rot_dim = rot_dim;
    a.num_q_heads = num_q_heads;
    a.bf16 = dtype == KVQ_BF16;
    a.interleaved = interleaved != 0;
    a.scale = (fmt == KVQ_INT8 || fmt == KVQ_INT4) ? nullptr : scale;
    a.err = err;
    return kvq::launch_append_rotary(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

size_t kvq_verify_workspace_size(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                 int32_t max_query_len, int32_t max_context_len, int32_t fmt) {
    if (batch <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || max_query_len <= 0 || max_context_len <= 0) return 0;
    if (num_q_heads % num_kv_heads || num_q_heads / num_kv_heads > 8 || max_query_len > kvq::kMaxVerifyQuery) return 0;
    if (batch > kMaxBatch || max_context_len > 1 << 30 || (head_dim != 64 && head_dim != 128)) return 0;
    if (fmt != KVQ_E4M3 && fmt != KVQ_E5M2 && fmt != KVQ_INT8 && fmt != KVQ_INT4) return 0;
    int dev = 0;
    if (!current_device(&dev)) dev = 0;
    size_t most = 0;   // with and without group scales
    for (int ng = 1; ng <= (fmt == KVQ_INT8 || fmt == KVQ_INT4 ? 2 : 1); ++ng) {
        const kvq::VerifyPlan p = kvq::plan_verify(batch, num_q_heads, num_kv_heads, head_dim, ng, max_query_len,
                                                   max_context_len, sm_count(dev));
        most = std::max(most, kvq::verify_ws_bytes(p.teams, p.rows, head_dim));
    }
    return most;
}

kvq_status kvq_verify_attention(const void* q, const kvq_cache* cache, const int32_t* block_tables,
                                int32_t max_blocks_per_seq, const int32_t* context_lens, const int32_t* query_start,
                                const uint64_t* tree_mask, int32_t batch, int64_t num_q_tokens, int32_t num_q_heads,
                                int32_t max_query_len, int32_t max_context_len, const float* scale, int32_t fmt,
                                float sm_scale, void* out, void* workspace, size_t workspace_bytes,
                                kvq_stream_t stream) {
    kvq_status st = check_cache(cache, fmt);
    if (st != KVQ_OK) return st;
    if (batch < 0 || num_q_tokens < 0 || num_q_heads <= 0 || max_query_len < 0 || max_context_len < 0 ||
        max_blocks_per_seq <= 0)
        return KVQ_ERR_INVALID_ARG;
    if (num_q_heads % cache->num_kv_heads) return KVQ_ERR_INVALID_ARG;
    if (num_q_heads / cache->num_kv_heads > 8 || max_query_len > kvq::kMaxVerifyQuery || batch > kMaxBatch ||
        max_context_len > 1 << 30 || num_q_tokens > 0x7FFFFFFFll)
        return KVQ_ERR_UNSUPPORTED;
    if (batch == 0 || max_query_len == 0 || num_q_tokens == 0 || max_context_len == 0) return KVQ_OK;
    if (!q || !block_tables || !context_lens || !query_start || !out || !aligned(q, 16) || !aligned(out, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(query_start, 4) || !aligned(tree_mask, 8))
        return KVQ_ERR_INVALID_ARG;
    if (scale && !aligned(scale, 4)) return KVQ_ERR_INVALID_ARG;
    if (!(sm_scale >= 0.f) || std::isinf(sm_scale)) return KVQ_ERR_INVALID_ARG;
    int dev;
    const bool have = current_device(&dev);
    const kvq::VerifyPlan p = kvq::plan_verify(batch, num_q_heads, cache->num_kv_heads, cache->head_dim,
                                               view(cache).ngroups, max_query_len, max_context_len,
                                               sm_count(have ? dev : 0));
    if ((int64_t)batch * cache->num_kv_heads * p.row_tiles * ((max_context_len + 31) / 32) >= 0x7FFFFFFFll)
        return KVQ_ERR_UNSUPPORTED;   // flat tile indices are 32-bit
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < kvq::verify_ws_bytes(p.teams, p.rows, cache->head_dim))
        return KVQ_ERR_WORKSPACE;
    unsigned long long* err = have ? err_word(dev) : nullptr;
    if (!err) return KVQ_ERR_CUDA;
    kvq::VerifyArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.cache = view(cache);
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start = query_start;
    a.tree_mask = reinterpret_cast<const unsigned long long*>(tree_mask);
    a.num_q_tokens = num_q_tokens;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.batch = batch;
    a.num_q_heads = num_q_heads;
    a.max_query_len = max_query_len;
    a.max_context_len = max_context_len;
    a.scale = (fmt == KVQ_INT8 || fmt == KVQ_INT4) ? nullptr : scale;
    a.sm_scale = sm_scale > 0.f ? sm_scale : 1.0f / std::sqrt((float)cache->head_dim);
    a.out = static_cast<uint16_t*>(out);
    a.ws = static_cast<uint8_t*>(workspace);
    a.err = err;
    return kvq::launch_verify(a, p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_move_rows(const kvq_cache* cache, const int64_t* src_slots, const int64_t* dst_slots,
                         const int32_t* move_start, int32_t batch, int64_t num_moves, int32_t max_moves, int32_t fmt,
                         kvq_stream_t stream) {
    kvq_status st = check_cache(cache, fmt);
    if (st != KVQ_OK) return st;
    if (batch < 0 || num_moves < 0 || max_moves < 0) return KVQ_ERR_INVALID_ARG;
    if (max_moves > kvq::kMaxMoves || batch > 65535 || num_moves > 0x7FFFFFFFll) return KVQ_ERR_UNSUPPORTED;
    if (batch == 0 || num_moves == 0 || max_moves == 0) return KVQ_OK;
    if (!src_slots || !dst_slots || !move_start || !aligned(src_slots, 8) || !aligned(dst_slots, 8) ||
        !aligned(move_start, 4))
        return KVQ_ERR_INVALID_ARG;
    int dev;
    if (!current_device(&dev)) return KVQ_ERR_CUDA;
    unsigned long long* err = err_word(dev);
    if (!err) return KVQ_ERR_CUDA;
    kvq::MoveArgs a{view(cache), src_slots, dst_slots, move_start, num_moves, batch, max_moves, err};
    return kvq::launch_move(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_dequant(const kvq_cache* cache, const int64_t* slots, int64_t num_slots, const float* scale,
                       int32_t fmt, float* out_k, float* out_v, kvq_stream_t stream) {
    kvq_status st = check_cache(cache, fmt);
    if (st != KVQ_OK) return st;
    if (num_slots < 0) return KVQ_ERR_INVALID_ARG;
    if (num_slots == 0) return KVQ_OK;
    if (!slots || !out_k || !out_v || !aligned(slots, 8) || !aligned(out_k, 16) || !aligned(out_v, 16))
        return KVQ_ERR_INVALID_ARG;
    if (scale && !aligned(scale, 4)) return KVQ_ERR_INVALID_ARG;
    if (num_slots * cache->num_kv_heads * (cache->head_dim / 16) / 256 >= 0x7FFFFFFFll) return KVQ_ERR_UNSUPPORTED;
    int dev;
    if (!current_device(&dev)) return KVQ_ERR_CUDA;
    unsigned long long* err = err_word(dev);
    if (!err) return KVQ_ERR_CUDA;
    kvq::DequantArgs a{view(cache), slots, num_slots, (fmt == KVQ_INT8 || fmt == KVQ_INT4) ? nullptr : scale, out_k, out_v, err};
    return kvq::launch_dequant(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_encode_fp8(const float* x, void* codes, int64_t n, int32_t fmt, kvq_stream_t stream) {
    if (fmt != KVQ_E4M3 && fmt != KVQ_E5M2) return KVQ_ERR_INVALID_ARG;
    if (n < 0) return KVQ_ERR_INVALID_ARG;
    if (n == 0) return KVQ_OK;
    if (!x || !codes || !aligned(x, 16) || !aligned(codes, 16)) return KVQ_ERR_INVALID_ARG;
    return kvq::launch_encode_fp8(x, static_cast<uint8_t*>(codes), n, fmt,
                                  reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KVQ_OK
               : KVQ_ERR_CUDA;
}

kvq_status kvq_device_error_check(kvq_stream_t stream, int64_t* detail) {
    int dev;
    if (!current_device(&dev)) return KVQ_ERR_CUDA;
    unsigned long long* err = err_word(dev);
    if (!err) return KVQ_ERR_CUDA;
    if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return KVQ_ERR_CUDA;
    unsigned long long v = 0;
    if (cudaMemcpy(&v, err, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return KVQ_ERR_CUDA;
    if (v == 0) {
        if (detail) *detail = 0;
        return KVQ_OK;
    }
    const unsigned long long zero = 0;
    if (cudaMemcpy(err, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess) return KVQ_ERR_CUDA;
    int64_t d = (int64_t)(v & 0x00FFFFFFFFFFFFFFull);
    if (d & 0x0080000000000000ll) d |= (int64_t)0xFF00000000000000ull;  // sign-extend 56 bits
    if (detail) *detail = d;
    return (v >> 56) == kvq::DEV_ERR_TIMEOUT ? KVQ_ERR_TIMEOUT : KVQ_ERR_OUT_OF_RANGE;
}

}  // extern "C"
