// Host side of the C ABI in include/gdn_attention.h: config validation,
// argument checks and launches.
#include <algorithm>
#include <cmath>
#include <new>

#include "gdn_attention.h"
#include "gdn_attn.cuh"
#include "gdn_host.h"

using namespace gdn;

struct gdn_attn {
  gdn_attn_config cfg;
  int device, grid;
  unsigned char* ws;
};

namespace {

// The workspace: the error word, on lines of its own; the counters of tasks that several
// CTAs share; the plan, where there can be more requests than every CTA plans for itself; the
// parts' maxima and sums, and their outputs.
constexpr size_t kErrorBytes = 256;
constexpr size_t kPartRows = 256;            // most rows of a part with heads of up to 128
constexpr size_t kPartFloats = 256 * 128;    // floats of a part: as many rows, or half as many of 256
size_t up(size_t n) { return (n + 255) / 256 * 256; }
struct Layout {
  size_t done, seq, start, ml, part, end;
  Layout(const gdn_attn_config& c, int grid) {
    const size_t n = c.max_seqs > kAttnPlanned ? (size_t)c.max_seqs + 1 : 0;
    done = kErrorBytes;
    seq = done + up((size_t)grid * 8);
    start = seq + up(n * 16);
    ml = start + up(n * 8);
    part = ml + up((size_t)2 * grid * kPartRows * 8);
    end = part + (size_t)2 * grid * kPartFloats * 4;
  }
};

float scale_log2(const gdn_attn_config& c) { return (float)((double)c.scale * 1.4426950408889634); }

gdn_status validate(const gdn_attn_config* c) {
  if (!c) return GDN_ERR_ARG;
  if (c->num_q_heads <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0 || c->block_size <= 0 || c->max_tokens < 1 ||
      c->max_seqs < 1)
    return GDN_ERR_ARG;
  if (!std::isfinite(scale_log2(*c))) return GDN_ERR_ARG;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return GDN_ERR_UNSUPPORTED;
  if (c->num_q_heads % c->num_kv_heads != 0 || c->num_q_heads > 1024) return GDN_ERR_UNSUPPORTED;
  if (c->max_tokens > (1 << 24) || c->max_seqs > 65535) return GDN_ERR_UNSUPPORTED;
  if ((long long)c->max_tokens * (c->num_q_heads / c->num_kv_heads) > (1 << 30)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

gdn_status check_device(const gdn_attn* h) {
  int device;
  if (cudaGetDevice(&device) != cudaSuccess) return GDN_ERR_CUDA;
  return device == h->device ? GDN_OK : GDN_ERR_ARG;
}

const __nv_bfloat16* bf(const void* p) { return static_cast<const __nv_bfloat16*>(p); }

}  // namespace

// Tile map of rows of 64-column boxes, 128-byte swizzle, zeros outside: {columns, rows} or {columns, heads, tokens}.
bool gdn::attn_encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  typedef CUresult (*Fn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                         const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                         CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static Fn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return (Fn)f;
  }();
  const cuuint32_t one[3] = {1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool gdn::attn_row_map(CUtensorMap* m, const void* base, long long rows, long long cols, long long ld, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  return attn_encode(m, base, 2, dims, strides, box);
}

extern "C" size_t gdn_attn_workspace_bytes(const gdn_attn_config* cfg) {
  if (validate(cfg) != GDN_OK) return 0;
  return Layout(*cfg, sm_count()).end;
}

extern "C" gdn_status gdn_attn_create(const gdn_attn_config* cfg, void* workspace, size_t workspace_bytes, void* stream,
                                      gdn_attn_t** out) {
  if (!out) return GDN_ERR_ARG;
  *out = nullptr;
  const gdn_status st = validate(cfg);
  if (st != GDN_OK) return st;
  const int grid = sm_count();
  const Layout l(*cfg, grid);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < l.end) return GDN_ERR_ARG;
  int device;
  if (cudaGetDevice(&device) != cudaSuccess) return GDN_ERR_CUDA;
  if (cudaMemsetAsync(workspace, 0, l.seq, (cudaStream_t)stream) != cudaSuccess) return GDN_ERR_CUDA;
  gdn_attn* h = new (std::nothrow) gdn_attn{*cfg, device, grid, static_cast<unsigned char*>(workspace)};
  if (!h) return GDN_ERR_CUDA;
  *out = h;
  return GDN_OK;
}

extern "C" gdn_status gdn_attn_paged(gdn_attn_t* h, int32_t seqs, int32_t tokens, int32_t max_len, const void* q,
                                     int64_t ldq, const void* k_cache, int64_t ldk, const void* v_cache, int64_t ldv,
                                     int32_t num_blocks, const int32_t* block_table, int32_t max_blocks,
                                     const int32_t* cu_seqlens, const int32_t* context_lens, const void* gate, int64_t ldg,
                                     void* out, int64_t ldo, void* stream) {
  if (!h || seqs < 0 || tokens < 0 || max_len < 0 || num_blocks < 0 || max_blocks < 0) return GDN_ERR_ARG;
  const gdn_attn_config& c = h->cfg;
  if (seqs > c.max_seqs || tokens > c.max_tokens) return GDN_ERR_ARG;
  if (!cu_seqlens || !aligned(cu_seqlens, 4)) return GDN_ERR_ARG;
  if (seqs > 0 && (!context_lens || !aligned(context_lens, 4))) return GDN_ERR_ARG;
  if (seqs > 0 && max_blocks > 0 && (!block_table || !aligned(block_table, 4))) return GDN_ERR_ARG;
  if (tokens > 0 && (!q || !out)) return GDN_ERR_ARG;
  if (num_blocks > 0 && (!k_cache || !v_cache)) return GDN_ERR_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(gate, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return GDN_ERR_ARG;
  const long long cols = (long long)c.num_q_heads * c.head_dim, kv = (long long)c.num_kv_heads * c.head_dim;
  if (ldq < cols || ldo < cols || (gate && ldg < cols) || ldk < kv || ldv < kv) return GDN_ERR_ARG;
  if (ldq % 8 || ldo % 8 || (gate && ldg % 8) || ldk % 8 || ldv % 8) return GDN_ERR_ARG;
  const long long slots = (long long)num_blocks * c.block_size;
  if (slots > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  if (ldq >= (1LL << 38) || ldk >= (1LL << 38) || ldv >= (1LL << 38)) return GDN_ERR_UNSUPPORTED;  // a tile map's largest stride
  const Layout l(c, h->grid);
  const Span o = matrix(out, tokens, ldo, cols);
  const Span in[] = {matrix(q, tokens, ldq, cols), matrix(gate, tokens, ldg, cols), matrix(k_cache, slots, ldk, kv),
                     matrix(v_cache, slots, ldv, kv), {block_table, (size_t)seqs * max_blocks * 4},
                     {cu_seqlens, (size_t)(seqs + 1) * 4}, {context_lens, (size_t)seqs * 4}, {h->ws, l.end}};
  if (overlaps_any(o, in)) return GDN_ERR_ARG;
  const gdn_status st = check_device(h);
  if (st != GDN_OK) return st;
  if (tokens == 0) return GDN_OK;
  AttnParams p{};
  p.cu = cu_seqlens;
  p.ctx = context_lens;
  p.table = block_table;
  p.seqs = seqs;
  p.tokens = tokens;
  p.max_len = std::min(max_len, tokens);
  p.max_blocks = max_blocks;
  p.num_blocks = num_blocks;
  // positions stay below 2^31 with room for a tile past the last
  p.limit = (int)std::min((long long)max_blocks * c.block_size, (long long)INT32_MAX - 1024);
  p.block = FastDiv::of(c.block_size);
  p.group = FastDiv::of(c.num_q_heads / c.num_kv_heads);
  p.Hkv = c.num_kv_heads;
  p.q = bf(q);
  p.ldq = ldq;
  p.k = bf(k_cache);
  p.ldk = ldk;
  p.v = bf(v_cache);
  p.ldv = ldv;
  p.gate = bf(gate);
  p.ldg = ldg;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ldo = ldo;
  p.wide_out = aligned(out, 32) && ldo % 16 == 0;
  p.scale_log2 = scale_log2(c);
  p.scale_pow2 = p.scale_log2 > 0.f ? std::ldexp(1.f, std::ilogb(p.scale_log2)) : 0.f;
  p.error = reinterpret_cast<unsigned int*>(h->ws);
  p.done = reinterpret_cast<unsigned int*>(h->ws + l.done);
  p.part = reinterpret_cast<float*>(h->ws + l.part);
  p.part_ml = reinterpret_cast<float2*>(h->ws + l.ml);
  if (c.max_seqs > kAttnPlanned) {  // room for the plan; the launchers say whether it is made there
    p.seq = reinterpret_cast<int4*>(h->ws + l.seq);
    p.start = reinterpret_cast<long long*>(h->ws + l.start);
  }
  // Rows of a request and key/value head: a tile of 16 has them all, or the tensor cores' tiles (which
  // hold a token's heads together, and need a cache to map). These take a row's maximum and hide keys before they scale,
  // which is right for scales above zero alone; the few rows' form scales first. Single tokens, few rows' form and
  // tiles: 64 over up to 8192, 64 heads of 128 on 8, 162 and 214 us; 8 heads on 1, 32 and 38; 8 over up to 30000 81 and 85;
  // 64 over up to 4096, heads of 64, 24 and 35; heads of 256, 48 over up to 8192, 132 and 121. 20 rows are in gdn_attn_rows.cu.
  const bool few = (long long)p.max_len * p.group.d <= 16 || p.group.d > 128 || num_blocks == 0 || !(p.scale_log2 > 0.f);
  return cuda_status((few ? launch_attn_rows : launch_attn_tiles)(p, c.head_dim, h->grid, (cudaStream_t)stream));
}

extern "C" gdn_status gdn_attn_check(gdn_attn_t* h, void* stream, uint32_t* detail) {
  if (!h) return GDN_ERR_ARG;
  const gdn_status st = check_device(h);
  if (st != GDN_OK) return st;
  uint32_t word = 0;
  if (cudaMemcpyAsync(&word, h->ws, 4, cudaMemcpyDeviceToHost, (cudaStream_t)stream) != cudaSuccess ||
      cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (detail) *detail = word;
  if (!word) return GDN_OK;
  const uint32_t s = word >> 24;
  return s == GDN_ERR_DEADLINE || s == GDN_ERR_INDEX ? (gdn_status)s : GDN_ERR_FAILED;
}

extern "C" gdn_status gdn_attn_reset(gdn_attn_t* h, void* stream) {
  if (!h) return GDN_ERR_ARG;
  const gdn_status st = check_device(h);
  if (st != GDN_OK) return st;
  return cuda_status(cudaMemsetAsync(h->ws, 0, Layout(h->cfg, h->grid).seq, (cudaStream_t)stream));
}

extern "C" void gdn_attn_destroy(gdn_attn_t* h) { delete h; }

extern "C" gdn_status gdn_kv_append(int32_t tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                    const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                                    const int32_t* token_pos, const int64_t* slots, int64_t num_slots,
                                    const float* inv_freq, int32_t rotary_dim, int32_t interleaved, const void* q_norm_w,
                                    const void* k_norm_w, float norm_eps, void* q_out, int64_t ldqo, void* k_cache,
                                    int64_t ldkc, void* v_cache, int64_t ldvc, uint32_t* error, void* stream) {
  if (tokens < 0 || num_kv_heads <= 0 || num_slots < 0 || rotary_dim < 0 || !q != !q_out) return GDN_ERR_ARG;
  if (!q) num_q_heads = 0;
  if (q && num_q_heads <= 0) return GDN_ERR_ARG;
  if (!(norm_eps >= 0.f) || rotary_dim > head_dim || (rotary_dim > 0 && !inv_freq)) return GDN_ERR_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return GDN_ERR_UNSUPPORTED;
  if (rotary_dim % 16 || num_q_heads > 65536 || num_kv_heads > 65536) return GDN_ERR_UNSUPPORTED;
  const long long cols = (long long)num_q_heads * head_dim, kv = (long long)num_kv_heads * head_dim;
  if ((q && (ldq < cols || ldqo < cols || ldq % 8 || ldqo % 8)) || ldk < kv || ldv < kv || ldkc < kv || ldvc < kv ||
      ldk % 8 || ldv % 8 || ldkc % 8 || ldvc % 8)
    return GDN_ERR_ARG;
  if (tokens == 0) return GDN_OK;
  if (!k || !v || !token_pos || !slots || (num_slots > 0 && (!k_cache || !v_cache))) return GDN_ERR_ARG;
  const void* a16[] = {q, k, v, q_norm_w, k_norm_w, q_out, k_cache, v_cache};
  for (const void* a : a16)
    if (!aligned(a, 16)) return GDN_ERR_ARG;
  if (!aligned(token_pos, 4) || !aligned(slots, 8) || !aligned(inv_freq, 4) || !aligned(error, 4)) return GDN_ERR_ARG;
  const Span outs[] = {matrix(q_out, tokens, ldqo, cols), matrix(k_cache, num_slots, ldkc, kv),
                       matrix(v_cache, num_slots, ldvc, kv), {error, error ? (size_t)4 : 0}};
  const Span in[] = {matrix(k, tokens, ldk, kv), matrix(v, tokens, ldv, kv), {token_pos, (size_t)tokens * 4},
                     {slots, (size_t)tokens * 8}, {inv_freq, (size_t)rotary_dim * 2},
                     {q_norm_w, q_norm_w ? (size_t)head_dim * 2 : 0}, {k_norm_w, k_norm_w ? (size_t)head_dim * 2 : 0}};
  const Span qs = matrix(q, tokens, ldq, cols);
  for (int i = 0; i < 4; ++i) {
    if (overlaps_any(outs[i], in)) return GDN_ERR_ARG;
    if (overlap(outs[i], qs) && !(i == 0 && q == q_out && ldq == ldqo)) return GDN_ERR_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return GDN_ERR_ARG;
  }
  AppendParams p{};
  p.tokens = tokens;
  p.Hq = num_q_heads;
  p.Hkv = num_kv_heads;
  p.rotary = rotary_dim;
  p.q = bf(q);
  p.ldq = ldq;
  p.k = bf(k);
  p.ldk = ldk;
  p.v = bf(v);
  p.ldv = ldv;
  p.pos = token_pos;
  p.slots = reinterpret_cast<const long long*>(slots);
  p.num_slots = num_slots;
  p.freq = inv_freq;
  p.qw = bf(q_norm_w);
  p.kw = bf(k_norm_w);
  p.eps = norm_eps;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.ldqo = ldqo;
  p.k_cache = static_cast<__nv_bfloat16*>(k_cache);
  p.ldkc = ldkc;
  p.v_cache = static_cast<__nv_bfloat16*>(v_cache);
  p.ldvc = ldvc;
  p.error = error;
  return cuda_status(launch_kv_append(p, head_dim, interleaved != 0, (cudaStream_t)stream));
}
