// api.cu -- host side of the C ABI declared in include/unstep.h: argument validation, cache
// metadata, the RoPE coefficient tables, window resolution, TMA descriptors and launches.
//
// UnStep paper (arXiv 2609.32518), abstract: RoPE from precomputed coefficients, KV indexing and
// a limited temporal window of the attention KV cache; Table 3: chunks of three latent frames.
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <vector>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "../../include/unstep.h"
#include "block_norm.h"
#include "conv3d.h"
#include "gemm.h"
#include "internal.h"

namespace {

constexpr int kInitMagic = 0x55535450;    // "USTP": an initialised bf16 cache
constexpr int kInitMagicQ8 = 0x55535138;  // "USQ8": the base of an initialised 8-bit cache

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Stream and head extents of the activation tensors the cache's shard lives in.
int act_B(const unstep_cache_t *c) { return c->act_B > 0 ? c->act_B : c->B; }
int act_H(const unstep_cache_t *c) { return c->act_H > 0 ? c->act_H : c->H; }

// Shape fields only (no pointers): 0 if valid, else a status code.
int check_shape(const unstep_cache_t *c) {
  if (!c) return UNSTEP_ERR_ARG;
  if (c->B < 1 || c->H < 1 || c->Hg < 1 || c->Wg < 1 || c->cap_frames < 1 || c->max_pos_t < 1)
    return UNSTEP_ERR_ARG;
  if (c->d_t < 0 || c->d_h < 0 || c->d_w < 0 || (c->d_t & 1) || (c->d_h & 1) || (c->d_w & 1))
    return UNSTEP_ERR_ARG;
  if (c->d_t + c->d_h + c->d_w != c->D) return UNSTEP_ERR_ARG;
  if (!(c->theta > 0.0) || !std::isfinite(c->theta)) return UNSTEP_ERR_ARG;
  if (c->D != 64 && c->D != 128) return UNSTEP_ERR_UNSUPPORTED;
  // row and element indices of the kernels: rows per (b, h) and TMA extents fit in int32,
  // every element offset in int64
  const long long tf = static_cast<long long>(c->Hg) * c->Wg;
  const long long rows = tf * c->cap_frames;
  if (tf > (1ll << 24) || rows > (1ll << 30) || static_cast<long long>(c->B) * c->H > (1ll << 30))
    return UNSTEP_ERR_UNSUPPORTED;
  if (c->max_pos_t > (1 << 24)) return UNSTEP_ERR_UNSUPPORTED;
  // the shard's place in the activations
  const long long act_b = act_B(c), act_h = act_H(c);
  if (c->act_B < 0 || c->act_H < 0 || c->b0 < 0 || c->h0 < 0) return UNSTEP_ERR_ARG;
  if (c->b0 + static_cast<long long>(c->B) > act_b || c->h0 + static_cast<long long>(c->H) > act_h)
    return UNSTEP_ERR_ARG;
  if (act_b * act_h > (1ll << 30)) return UNSTEP_ERR_UNSUPPORTED;
  return UNSTEP_OK;
}

size_t table_floats(const unstep_cache_t *c) {
  return 2ull * (static_cast<size_t>(c->max_pos_t) * (c->d_t / 2) +
                 static_cast<size_t>(c->Hg) * (c->d_h / 2) +
                 static_cast<size_t>(c->Wg) * (c->d_w / 2));
}

// Initialised as a bf16 cache or as the base of an 8-bit one (host-side plans take both).
bool is_initialized(const unstep_cache_t *c) {
  return c->initialized == kInitMagic || c->initialized == kInitMagicQ8;
}

int check_ready(const unstep_cache_t *c) {
  int rc = check_shape(c);
  if (rc) return rc;
  if (c->initialized != kInitMagic) return UNSTEP_ERR_ARG;
  if (!c->k_cache || !c->v_cache || !c->slot_frame || !c->cos_sin || !c->dev_error)
    return UNSTEP_ERR_ARG;
  return UNSTEP_OK;
}

// cuTensorMapEncodeTiled from the driver, fetched once through the runtime (no libcuda link).
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// bf16 tensor map with 128-byte swizzle: dims[0] is the contiguous channel axis (boxed 64 wide).
bool encode_bf16(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims,
                 const cuuint64_t *strides_bytes, const cuuint32_t *box) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank),
                  const_cast<void *>(base), dims, strides_bytes, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Multiprocessor count of the current device (cached per device).
int device_sms() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev >= 0 && dev < 64) {
    int v = cache[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev >= 0 && dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

long long max_units(const unstep_cache_t *c) {
  const long long rows = static_cast<long long>(c->cap_frames) * c->Hg * c->Wg;
  return static_cast<long long>(c->B) * c->H * ((rows + 255) / 256);
}

size_t scratch_bytes_for(const unstep_cache_t *c, int sms) {
  return unstep::attn_counter_bytes(max_units(c)) +
         2ull * static_cast<size_t>(sms) * unstep::attn_slot_floats(c->D) * sizeof(float);
}

// ---- checkpoint buffer header (layout documented with unstep_cache_save) ----
constexpr int kStateMagic = 0x43545355;    // "USTC"
constexpr int kStateMagicQ8 = 0x51545355;  // "USTQ": an 8-bit cache
constexpr int kStateVersion = 1;
constexpr size_t kStateSlotOffset = 128;

size_t state_header_bytes(const unstep_cache_t *c) {
  return kStateSlotOffset + ((sizeof(int) * static_cast<size_t>(c->cap_frames) + 15) / 16) * 16;
}

void put_i32(unsigned char *p, size_t off, int v) { std::memcpy(p + off, &v, sizeof(int)); }
int get_i32(const unsigned char *p, size_t off) {
  int v;
  std::memcpy(&v, p + off, sizeof(int));
  return v;
}

void write_state_header(const unstep_cache_t *c, int magic, unsigned char *p) {
  const int f[14] = {c->B,  c->H,          c->D,         c->Hg,  c->Wg,  c->d_t, c->d_h,
                     c->d_w, c->cap_frames, c->max_pos_t, act_B(c), act_H(c), c->b0, c->h0};
  put_i32(p, 0, magic);
  put_i32(p, 4, kStateVersion);
  for (int i = 0; i < 14; ++i) put_i32(p, 8 + 4 * i, f[i]);
  std::memcpy(p + 64, &c->theta, sizeof(double));
  put_i32(p, 72, c->frames_written);
  put_i32(p, 76, c->first_frame);
  put_i32(p, 80, c->last_chunk_start);
  put_i32(p, 84, c->last_chunk_frames);
}

int read_state_header(const unsigned char *p, int magic, unstep_cache_t *c) {
  if (get_i32(p, 0) != magic || get_i32(p, 4) != kStateVersion) return UNSTEP_ERR_ARG;
  int *f[14] = {&c->B,  &c->H,          &c->D,         &c->Hg,    &c->Wg,    &c->d_t, &c->d_h,
                &c->d_w, &c->cap_frames, &c->max_pos_t, &c->act_B, &c->act_H, &c->b0,  &c->h0};
  for (int i = 0; i < 14; ++i) *f[i] = get_i32(p, 8 + 4 * i);
  std::memcpy(&c->theta, p + 64, sizeof(double));
  c->frames_written = get_i32(p, 72);
  c->first_frame = get_i32(p, 76);
  c->last_chunk_start = get_i32(p, 80);
  c->last_chunk_frames = get_i32(p, 84);
  return UNSTEP_OK;
}

// Shape and shard identical (the metadata may differ).
bool same_state_shape(const unstep_cache_t *a, const unstep_cache_t *b) {
  return a->B == b->B && a->H == b->H && a->D == b->D && a->Hg == b->Hg && a->Wg == b->Wg &&
         a->d_t == b->d_t && a->d_h == b->d_h && a->d_w == b->d_w &&
         a->cap_frames == b->cap_frames && a->max_pos_t == b->max_pos_t &&
         act_B(a) == act_B(b) && act_H(a) == act_H(b) && a->b0 == b->b0 && a->h0 == b->h0 &&
         std::memcmp(&a->theta, &b->theta, sizeof(double)) == 0;
}

// What unstep_cache_init and unstep_q8_cache_init share: checks, coefficient tables, `kvb` zeroed
// bytes of each of K and V, slots, counters and metadata.
int init_cache(unstep_cache_t *cache, size_t kvb, int magic, cudaStream_t s) {
  int rc = check_shape(cache);
  if (rc) return rc;
  if (!cache->k_cache || !cache->v_cache || !cache->slot_frame || !cache->cos_sin ||
      !cache->dev_error)
    return UNSTEP_ERR_ARG;
  if (!aligned16(cache->k_cache) || !aligned16(cache->v_cache) || !aligned16(cache->cos_sin) ||
      !aligned16(cache->attn_scratch))
    return UNSTEP_ERR_ALIGN;
  if (cache->attn_scratch) {
    const int sms = device_sms();
    if (sms <= 0) return UNSTEP_ERR_CUDA;
    if (cache->attn_scratch_bytes < scratch_bytes_for(cache, sms)) return UNSTEP_ERR_ARG;
  }
  // cached coefficients: cos/sin of pos * theta^(-2j/d_a), computed in fp64, stored fp32
  std::vector<float> tab(table_floats(cache));
  size_t o = 0;
  const int dims[3] = {cache->d_t, cache->d_h, cache->d_w};
  const int npos[3] = {cache->max_pos_t, cache->Hg, cache->Wg};
  for (int a = 0; a < 3; ++a) {
    const int half = dims[a] / 2;
    for (int pos = 0; pos < npos[a]; ++pos) {
      for (int j = 0; j < half; ++j) {
        const double inv = std::pow(cache->theta, -2.0 * j / static_cast<double>(dims[a]));
        const double ang = static_cast<double>(pos) * inv;
        tab[o++] = static_cast<float>(std::cos(ang));
        tab[o++] = static_cast<float>(std::sin(ang));
      }
    }
  }
  if (cudaMemcpyAsync(cache->cos_sin, tab.data(), tab.size() * sizeof(float),
                      cudaMemcpyHostToDevice, s) != cudaSuccess ||
      cudaMemsetAsync(cache->k_cache, 0, kvb, s) != cudaSuccess ||
      cudaMemsetAsync(cache->v_cache, 0, kvb, s) != cudaSuccess ||
      cudaMemsetAsync(cache->slot_frame, 0xFF, sizeof(int) * cache->cap_frames, s) !=
          cudaSuccess ||
      cudaMemsetAsync(cache->dev_error, 0, sizeof(int), s) != cudaSuccess ||
      (cache->attn_scratch &&
       cudaMemsetAsync(cache->attn_scratch, 0, unstep::attn_counter_bytes(max_units(cache)), s) !=
           cudaSuccess)) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  cache->frames_written = 0;
  cache->first_frame = 0;
  cache->last_chunk_start = -1;
  cache->last_chunk_frames = 0;
  cache->initialized = magic;
  return UNSTEP_OK;
}

// Launch parameters of an append, all but the queries.
unstep::RopeAppendParams append_params(const unstep_cache_t *cache, const void *k, const void *v,
                                       int frame_idx, unstep_grid_t grid) {
  unstep::RopeAppendParams p{};
  p.k = k;
  p.v = v;
  p.k_cache = cache->k_cache;
  p.v_cache = cache->v_cache;
  p.slot_frame = cache->slot_frame;
  const float2 *tab = reinterpret_cast<const float2 *>(cache->cos_sin);
  p.tab_t = tab;
  p.tab_h = p.tab_t + static_cast<size_t>(cache->max_pos_t) * (cache->d_t / 2);
  p.tab_w = p.tab_h + static_cast<size_t>(cache->Hg) * (cache->d_h / 2);
  p.B = cache->B;
  p.H = cache->H;
  p.act_H = act_H(cache);
  p.b0 = cache->b0;
  p.h0 = cache->h0;
  p.sharded = (p.act_H != p.H || p.b0 != 0 || p.h0 != 0) ? 1 : 0;
  p.D = cache->D;
  p.Hg = cache->Hg;
  p.Wg = cache->Wg;
  p.Tf = cache->Hg * cache->Wg;
  p.L = grid.frames * p.Tf;
  p.half_t = cache->d_t / 2;
  p.half_h = cache->d_h / 2;
  p.half_w = cache->d_w / 2;
  p.frame_idx = frame_idx;
  p.frames = grid.frames;
  p.cap = cache->cap_frames;
  p.rows = cache->cap_frames * p.Tf;
  p.act_B = act_B(cache);
  p.max_pos_t = cache->max_pos_t;
  p.dev_error = cache->dev_error;
  return p;
}

// Metadata after an append was launched.
void note_append(unstep_cache_t *cache, int frame_idx, int frames, bool is_new) {
  if (is_new) {
    if (cache->last_chunk_frames == 0) cache->first_frame = frame_idx;
    cache->frames_written = frame_idx + frames;
  }
  cache->last_chunk_start = frame_idx;
  cache->last_chunk_frames = frames;
}

unsigned next_epoch() {
  static std::atomic<unsigned> counter{0};
  return counter.fetch_add(1, std::memory_order_relaxed) % 0xFFFFFFu + 1u;
}

}  // namespace

extern "C" {

int unstep_version(void) { return 101; }

const char *unstep_status_string(int status) {
  switch (status) {
    case UNSTEP_OK: return "ok";
    case UNSTEP_ERR_ARG: return "invalid argument";
    case UNSTEP_ERR_SHAPE: return "shape mismatch";
    case UNSTEP_ERR_ALIGN: return "pointer not 16-byte aligned";
    case UNSTEP_ERR_FRAME_ORDER: return "frame_idx is neither the next chunk nor the latest chunk";
    case UNSTEP_ERR_WINDOW: return "window outside [chunk frames, cache capacity] or empty cache";
    case UNSTEP_ERR_UNSUPPORTED: return "unsupported head width or size";
    case UNSTEP_ERR_CUDA: return "CUDA runtime error";
    case UNSTEP_ERR_DEVICE_TIMEOUT: return "a device-side wait timed out";
    case UNSTEP_ERR_SCRATCH_LIMIT:
      return "the call needs more scratch than the library's fixed device buffer holds";
    case UNSTEP_ERR_DEVICE_BOUNDS:
      return "a device-side index check failed (debug build)";
    default: return "unknown status";
  }
}

size_t unstep_cache_table_bytes(const unstep_cache_t *cache) {
  if (check_shape(cache)) return 0;
  return table_floats(cache) * sizeof(float);
}

size_t unstep_cache_kv_bytes(const unstep_cache_t *cache) {
  if (check_shape(cache)) return 0;
  return static_cast<size_t>(cache->B) * cache->H * cache->cap_frames * cache->Hg * cache->Wg *
         cache->D * 2;
}

size_t unstep_attn_scratch_bytes(const unstep_cache_t *cache) {
  if (check_shape(cache)) return 0;
  const int sms = device_sms();
  if (sms <= 0) return 0;
  return scratch_bytes_for(cache, sms);
}

int unstep_cache_init(unstep_cache_t *cache, unstep_stream_t stream) {
  // the base of an 8-bit cache has buffers of another size: unstep_q8_cache_init resets it
  if (cache && cache->initialized == kInitMagicQ8) return UNSTEP_ERR_ARG;
  return init_cache(cache, unstep_cache_kv_bytes(cache), kInitMagic,
                    reinterpret_cast<cudaStream_t>(stream));
}

int unstep_append_plan(const unstep_cache_t *cache, int frame_idx, unstep_grid_t grid,
                       int *slots_out) {
  int rc = check_shape(cache);
  if (rc) return rc;
  if (!is_initialized(cache)) return UNSTEP_ERR_ARG;
  if (grid.Hg != cache->Hg || grid.Wg != cache->Wg || grid.frames < 1) return UNSTEP_ERR_SHAPE;
  if (grid.frames > cache->cap_frames) return UNSTEP_ERR_WINDOW;
  if (frame_idx < 0 || static_cast<long long>(frame_idx) + grid.frames > cache->max_pos_t)
    return UNSTEP_ERR_ARG;
  int is_new;
  if (cache->last_chunk_frames == 0) {
    is_new = 1;  // the stream's first chunk may start at any temporal position
  } else if (frame_idx == cache->frames_written) {
    is_new = 1;
  } else if (frame_idx == cache->last_chunk_start && grid.frames == cache->last_chunk_frames) {
    is_new = 0;
  } else {
    return UNSTEP_ERR_FRAME_ORDER;
  }
  if (slots_out)
    for (int i = 0; i < grid.frames; ++i) slots_out[i] = (frame_idx + i) % cache->cap_frames;
  return is_new;
}

int unstep_rope_kv_append_ex(void *q, const void *k, const void *v, unstep_cache_t *cache,
                             int frame_idx, unstep_grid_t grid, unsigned flags,
                             unstep_stream_t stream) {
  int rc = check_ready(cache);
  if (rc) return rc;
  if (flags & ~static_cast<unsigned>(UNSTEP_APPEND_DEFER_Q_ROPE)) return UNSTEP_ERR_ARG;
  const bool rotate_q = !(flags & UNSTEP_APPEND_DEFER_Q_ROPE);
  if ((rotate_q && !q) || !k || !v) return UNSTEP_ERR_ARG;
  if ((rotate_q && !aligned16(q)) || !aligned16(k) || !aligned16(v)) return UNSTEP_ERR_ALIGN;
  const int is_new = unstep_append_plan(cache, frame_idx, grid, nullptr);
  if (is_new < 0) return is_new;
  unstep::RopeAppendParams p = append_params(cache, k, v, frame_idx, grid);
  p.q = rotate_q ? q : nullptr;
  p.rotate_q = rotate_q ? 1 : 0;
  if (unstep::launch_rope_kv_append(p, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  note_append(cache, frame_idx, grid.frames, is_new == 1);
  return UNSTEP_OK;
}

int unstep_rope_kv_append(void *q, const void *k, const void *v, unstep_cache_t *cache,
                          int frame_idx, unstep_grid_t grid, unstep_stream_t stream) {
  return unstep_rope_kv_append_ex(q, k, v, cache, frame_idx, grid, 0u, stream);
}

int unstep_window_plan(const unstep_cache_t *cache, int window, unstep_window_plan_t *plan) {
  int rc = check_shape(cache);
  if (rc) return rc;
  if (!plan || !is_initialized(cache)) return UNSTEP_ERR_ARG;
  if (cache->last_chunk_frames < 1) return UNSTEP_ERR_WINDOW;
  if (window < cache->last_chunk_frames || window > cache->cap_frames) return UNSTEP_ERR_WINDOW;
  const int tf = cache->Hg * cache->Wg;
  const int cap = cache->cap_frames;
  const int f_end = cache->last_chunk_start + cache->last_chunk_frames - 1;
  int f0 = f_end - window + 1;
  if (f0 < cache->first_frame) f0 = cache->first_frame;
  const int nf = f_end - f0 + 1;
  const int s0 = f0 % cap;
  plan->first_frame = f0;
  plan->last_frame = f_end;
  plan->keys = nf * tf;
  plan->seg_row[0] = s0 * tf;
  if (s0 + nf <= cap) {
    plan->seg_len[0] = nf * tf;
    plan->seg_row[1] = 0;
    plan->seg_len[1] = 0;
  } else {
    plan->seg_len[0] = (cap - s0) * tf;
    plan->seg_row[1] = 0;
    plan->seg_len[1] = (s0 + nf - cap) * tf;
  }
  return UNSTEP_OK;
}

}  // extern "C"

namespace {

// Whether `na` bytes at a and `nb` at b share one (a NULL shares none).
bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x && y && (x < y ? y - x < na : x - y < nb);
}

// Whether `bytes` at p share one with an 8-bit cache's codes or scales.
bool overlaps_rows(const void *p, size_t bytes, const unstep_q8_cache_t *c) {
  const size_t codes = unstep_q8_cache_kv_bytes(c), scales = unstep_q8_cache_scale_bytes(c);
  return overlap(p, bytes, c->base.k_cache, codes) || overlap(p, bytes, c->base.v_cache, codes) ||
         overlap(p, bytes, c->k_scale, scales) || overlap(p, bytes, c->v_scale, scales);
}

// Bytes of a tensor of `rows` tokens' activations.
size_t act_bytes(const unstep_cache_t *c, long long rows) {
  return 2ull * static_cast<size_t>(act_B(c)) * static_cast<size_t>(rows) *
         static_cast<size_t>(act_H(c)) * static_cast<size_t>(c->D);
}

// What unstep_window_attn_ex and unstep_window_attn_noalloc share: validation, the window plan,
// the tensor maps, the persistent schedule and the launch.  `fixed_buffer` selects the scratch:
// false, the cache's own (cache->attn_scratch, sized at unstep_cache_init; none: one CTA per
// unit); true, the library's fixed device buffer, whose counters are zeroed on `st` first.
// `q8`: the 8-bit cache whose base `cache` is, checked by the caller.
int window_attn_launch(const void *q, const unstep_cache_t *cache, int window, void *out,
                       unsigned flags, bool fixed_buffer, cudaStream_t st,
                       const unstep_q8_cache_t *q8 = nullptr) {
  int rc = q8 ? UNSTEP_OK : check_ready(cache);
  if (rc) return rc;
  if (flags & ~static_cast<unsigned>(UNSTEP_ATTN_ROPE_Q)) return UNSTEP_ERR_ARG;
  if (!q || !out) return UNSTEP_ERR_ARG;
  if (!aligned16(q) || !aligned16(out)) return UNSTEP_ERR_ALIGN;
  unstep_window_plan_t plan;
  rc = unstep_window_plan(cache, window, &plan);
  if (rc) return rc;
  const int D = cache->D, H = cache->H, B = cache->B;
  const int tf = cache->Hg * cache->Wg;
  const int L = cache->last_chunk_frames * tf;
  const long long R = static_cast<long long>(cache->cap_frames) * tf;
  // a unit's rows are written while other CTAs may still load its queries or the cache
  if (q8 && (overlap(out, act_bytes(cache, L), q, act_bytes(cache, L)) ||
             overlaps_rows(out, act_bytes(cache, L), q8)))
    return UNSTEP_ERR_ARG;
  const int n_pairs = (L + 255) / 256;
  // (head, 256-query) units are numbered in int32 by the kernel
  const long long units = static_cast<long long>(B) * H * n_pairs;
  if (units > INT_MAX) return fixed_buffer ? UNSTEP_ERR_SCRATCH_LIMIT : UNSTEP_ERR_UNSUPPORTED;
  const int U = static_cast<int>(units);

  void *scratch = nullptr;
  size_t counter_bytes = 0;
  int sms = 0;
  if (fixed_buffer) {
    size_t capacity = 0;
    if (unstep::static_attn_scratch(&scratch, &capacity) != cudaSuccess) {
      cudaGetLastError();
      return UNSTEP_ERR_CUDA;
    }
    sms = device_sms();
    if (sms <= 0) return UNSTEP_ERR_CUDA;
    counter_bytes = unstep::attn_counter_bytes(U);
    const size_t need = counter_bytes + 2ull * static_cast<size_t>(sms) *
                                            unstep::attn_slot_floats(D) * sizeof(float);
    if (need > capacity) return UNSTEP_ERR_SCRATCH_LIMIT;
  } else if (cache->attn_scratch) {
    scratch = cache->attn_scratch;
    counter_bytes = unstep::attn_counter_bytes(max_units(cache));
    sms = device_sms();
  }

  CUtensorMap tq, tk, tv;
  {
    // the whole activation tensor; the shard's streams and heads are TMA coordinates
    const cuuint64_t aB = static_cast<cuuint64_t>(act_B(cache));
    const cuuint64_t aH = static_cast<cuuint64_t>(act_H(cache));
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), aH, static_cast<cuuint64_t>(L), aB};
    const cuuint64_t str[3] = {static_cast<cuuint64_t>(D) * 2, aH * D * 2,
                               static_cast<cuuint64_t>(L) * aH * D * 2};
    const cuuint32_t box[4] = {64, 1, 128, 1};
    if (!encode_bf16(&tq, q, 4, dims, str, box)) return UNSTEP_ERR_CUDA;
  }
  if (!q8) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(R),
                                static_cast<cuuint64_t>(B) * H};
    const cuuint64_t str[2] = {static_cast<cuuint64_t>(D) * 2,
                               static_cast<cuuint64_t>(R) * D * 2};
    const cuuint32_t box[3] = {64, 128, 1};
    if (!encode_bf16(&tk, cache->k_cache, 3, dims, str, box)) return UNSTEP_ERR_CUDA;
    if (!encode_bf16(&tv, cache->v_cache, 3, dims, str, box)) return UNSTEP_ERR_CUDA;
  }
  unstep::AttnParams p{};
  p.out = out;
  p.dev_error = cache->dev_error;
  p.B = B;
  p.H = H;
  p.act_H = act_H(cache);
  p.act_B = act_B(cache);
  p.b0 = cache->b0;
  p.h0 = cache->h0;
  p.L = L;
  p.rows = static_cast<int>(R);
  p.n_pairs = n_pairs;
  p.n_units = U;
  for (int s = 0; s < 2; ++s) {
    p.seg_row[s] = plan.seg_row[s];
    p.seg_len[s] = plan.seg_len[s];
    p.seg_tiles[s] = (plan.seg_len[s] + 127) / 128;
  }
  p.n_tiles = p.seg_tiles[0] + p.seg_tiles[1];
  p.div_pairs = unstep::make_fastdiv(static_cast<uint32_t>(p.n_pairs));
  p.div_heads = unstep::make_fastdiv(static_cast<uint32_t>(H));
  if (scratch && sms > 0) {
    // persistent schedule: whole units in waves of `sms` CTAs, the remainder split along keys
    p.dp_waves = U / sms;
    const int tail = U - p.dp_waves * sms;
    p.u_tail0 = p.dp_waves * sms;
    p.w_tail = static_cast<long long>(tail) * p.n_tiles;
    long long gsk = tail > 0 ? static_cast<long long>(tail) * 8 : 0;  // at most ~8 pieces/unit
    if (gsk > sms) gsk = sms;
    if (gsk > p.w_tail) gsk = p.w_tail;
    // a piece of fewer than four key tiles costs more in its scratch slot and merge than it saves
    // (8-bit caches: 72 queries over 144 keys 16.4 -> 12.3 us, 312 over 936 37 -> 31 us); the bf16
    // schedule keeps its pieces, and with them its results' bits
    if (q8) {
      const long long most = static_cast<long long>(tail) * (p.n_tiles < 8 ? 1 : p.n_tiles / 4);
      if (gsk > most) gsk = most;
    }
    p.g_sk = static_cast<int>(gsk);
    p.grid = p.dp_waves > 0 ? sms : p.g_sk;
    p.counters = static_cast<unsigned *>(scratch);
    p.slots = reinterpret_cast<float *>(static_cast<char *>(scratch) + counter_bytes);
    p.slot_floats = static_cast<int>(unstep::attn_slot_floats(D));
    p.epoch = next_epoch();
  } else {
    // no scratch: one CTA per unit, nothing is split
    p.dp_waves = 1;
    p.grid = p.n_units;
    p.u_tail0 = p.n_units;
    p.g_sk = 0;
    p.w_tail = 0;
  }
  p.scale_log2 = static_cast<float>(1.4426950408889634073599 / std::sqrt(static_cast<double>(D)));
  p.wait_limit_ns = unstep::kWaitLimitNs;
  if (flags & UNSTEP_ATTN_ROPE_Q) {
    // q is the latest chunk's un-rotated queries: row l is token (i, y, x) of frame
    // last_chunk_start + i, rotated with the append's tables in the kernel's prologue
    const float2 *tab = reinterpret_cast<const float2 *>(cache->cos_sin);
    p.rope_q = 1;
    p.tab_t = tab;
    p.tab_h = p.tab_t + static_cast<size_t>(cache->max_pos_t) * (cache->d_t / 2);
    p.tab_w = p.tab_h + static_cast<size_t>(cache->Hg) * (cache->d_h / 2);
    p.half_t = cache->d_t / 2;
    p.half_h = cache->d_h / 2;
    p.half_w = cache->d_w / 2;
    p.Tf = tf;
    p.Wg = cache->Wg;
    p.frame0 = cache->last_chunk_start;
    p.frames = cache->last_chunk_frames;
    const size_t tab_bytes = sizeof(float2) * (static_cast<size_t>(p.frames) * p.half_t +
                                               static_cast<size_t>(cache->Hg) * p.half_h +
                                               static_cast<size_t>(cache->Wg) * p.half_w);
    p.tab_smem = tab_bytes <= static_cast<size_t>(unstep::kQRopeTabBytes) ? 1 : 0;
    p.div_tf = unstep::make_fastdiv(static_cast<uint32_t>(tf));
    p.div_wg = unstep::make_fastdiv(static_cast<uint32_t>(cache->Wg));
  }
  // the fixed buffer keeps whatever the previous call left in it: the counts must start at zero
  if (fixed_buffer && cudaMemsetAsync(scratch, 0, counter_bytes, st) != cudaSuccess) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  if (q8)
    p.q8 = unstep::Q8Rows{static_cast<const unsigned char *>(cache->k_cache),
                          static_cast<const unsigned char *>(cache->v_cache),
                          static_cast<const unsigned char *>(q8->k_scale),
                          static_cast<const unsigned char *>(q8->v_scale)};
  if ((q8 ? unstep::launch_q8_window_attn(D, tq, p, st)
          : unstep::launch_window_attn(D, tq, tk, tv, p, st)) != cudaSuccess) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  return UNSTEP_OK;
}

}  // namespace

extern "C" {

int unstep_window_attn_ex(const void *q, const unstep_cache_t *cache, int window, void *out,
                          unsigned flags, unstep_stream_t stream) {
  return window_attn_launch(q, cache, window, out, flags, false,
                            reinterpret_cast<cudaStream_t>(stream));
}

int unstep_window_attn(const void *q, const unstep_cache_t *cache, int window, void *out,
                       unstep_stream_t stream) {
  return unstep_window_attn_ex(q, cache, window, out, 0u, stream);
}

int unstep_window_attn_noalloc(const void *q, const unstep_cache_t *cache, int window,
                               void *out, unstep_stream_t stream) {
  return window_attn_launch(q, cache, window, out, 0u, true,
                            reinterpret_cast<cudaStream_t>(stream));
}

int unstep_gemm_bf16(const void *a, int lda, const void *b, int ldb, void *c, int ldc, int M,
                     int N, int K, int *dev_error, unstep_stream_t stream) {
  if (!a || !b || !c || !dev_error) return UNSTEP_ERR_ARG;
  if (M < 1 || N < 1 || K < 1) return UNSTEP_ERR_SHAPE;
  if ((N & 7) || (K & 7) || (lda & 7) || (ldb & 7) || (ldc & 7) || lda < K || ldb < K || ldc < N)
    return UNSTEP_ERR_SHAPE;
  if (!aligned16(a) || !aligned16(b) || !aligned16(c)) return UNSTEP_ERR_ALIGN;
  CUtensorMap ta, tb;
  {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(M)};
    const cuuint64_t str[1] = {static_cast<cuuint64_t>(lda) * 2};
    const cuuint32_t box[2] = {64, 128};
    if (!encode_bf16(&ta, a, 2, dims, str, box)) return UNSTEP_ERR_CUDA;
  }
  {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(N)};
    const cuuint64_t str[1] = {static_cast<cuuint64_t>(ldb) * 2};
    const cuuint32_t box[2] = {64, 128};
    if (!encode_bf16(&tb, b, 2, dims, str, box)) return UNSTEP_ERR_CUDA;
  }
  // CTA pairs (256 x 256 tiles) when the product is at least one pair tile; else single CTAs
#ifndef UNSTEP_GEMM_2SM
#define UNSTEP_GEMM_2SM 1
#endif
  const bool pair = UNSTEP_GEMM_2SM && M >= 256 && N >= 256;
  CUtensorMap tc;
  if (pair) {
    // the pair kernel stores C through TMA, one 64-column x 32-row box per epilogue warp
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
    const cuuint64_t str[1] = {static_cast<cuuint64_t>(ldc) * 2};
    const cuuint32_t box[2] = {64, 32};
    if (!encode_bf16(&tc, c, 2, dims, str, box)) return UNSTEP_ERR_CUDA;
  }
  const cudaError_t e =
      pair ? unstep::launch_gemm2sm_bf16_tn(ta, tb, tc, M, N, K, dev_error,
                                            reinterpret_cast<cudaStream_t>(stream))
           : unstep::launch_gemm_bf16_tn(ta, tb, c, M, N, K, ldc, dev_error,
                                         reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  return UNSTEP_OK;
}

int unstep_lowrank_linear(const void *x, const void *w1, const void *w2, void *t, void *y, int M,
                          int d_in, int rank, int d_out, int *dev_error, unstep_stream_t stream) {
  int rc = unstep_gemm_bf16(x, d_in, w1, d_in, t, rank, M, rank, d_in, dev_error, stream);
  if (rc) return rc;
  return unstep_gemm_bf16(t, rank, w2, rank, y, d_out, M, d_out, rank, dev_error, stream);
}

int unstep_renoise(const void *x0, const void *eps, void *out, long long n, float sigma,
                   unstep_stream_t stream) {
  if (!x0 || !eps || !out || n < 0) return UNSTEP_ERR_ARG;
  if (!(sigma >= 0.f && sigma <= 1.f)) return UNSTEP_ERR_ARG;
  if (!aligned16(x0) || !aligned16(eps) || !aligned16(out)) return UNSTEP_ERR_ALIGN;
  if (n == 0) return UNSTEP_OK;
  if (unstep::launch_renoise(x0, eps, out, n, sigma, reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  return UNSTEP_OK;
}

size_t unstep_conv3d_scratch_bytes(void) {
  const int sms = device_sms();
  if (sms <= 0) return 0;
  return unstep::conv_scratch_bytes(sms);
}

int unstep_conv3d_causal(const void *x, const void *w, const float *bias, void *y, int B, int T,
                         int H, int W, int C_in, int C_out, void *scratch, size_t scratch_bytes,
                         int *dev_error, unstep_stream_t stream) {
  if (!x || !w || !y || !dev_error) return UNSTEP_ERR_ARG;
  if (B < 1 || T < 1 || H < 1 || W < 1 || C_in < 1 || C_out < 1) return UNSTEP_ERR_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned16(scratch) ||
      (bias && (reinterpret_cast<uintptr_t>(bias) & 3u)))
    return UNSTEP_ERR_ALIGN;
  int sms = 0;
  if (scratch) {
    sms = device_sms();
    if (sms <= 0) return UNSTEP_ERR_CUDA;
    if (scratch_bytes < unstep::conv_scratch_bytes(sms)) return UNSTEP_ERR_ARG;
  }
  if (C_in % 64 != 0 || C_out % 8 != 0) return UNSTEP_ERR_UNSUPPORTED;
  const long long frames = static_cast<long long>(B) * (T + 2);
  const long long tiles_h = (H + unstep::kConvTileH - 1) / unstep::kConvTileH;
  const long long tiles_w = (W + 15) / 16;
  const long long m_tiles = static_cast<long long>(B) * T * tiles_h * tiles_w;
  const long long n_tiles = (C_out + 127) / 128;
  if (frames > 0x7FFFFFFFll || m_tiles * n_tiles > 0x7FFFFFFFll || W > (1 << 24) ||
      H > (1 << 24) || C_in > (1 << 16) || C_out > (1 << 24))
    return UNSTEP_ERR_UNSUPPORTED;
  CUtensorMap tmx, tmw;
  {
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(C_in), static_cast<cuuint64_t>(W),
                                static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(frames)};
    const cuuint64_t str[3] = {static_cast<cuuint64_t>(C_in) * 2,
                               static_cast<cuuint64_t>(W) * C_in * 2,
                               static_cast<cuuint64_t>(H) * W * C_in * 2};
    // the output tile's rows and a halo row on each side, for the three dy taps at once
    const cuuint32_t box[4] = {64, 16, static_cast<cuuint32_t>(unstep::kConvTileH + 2), 1};
    if (!encode_bf16(&tmx, x, 4, dims, str, box)) return UNSTEP_ERR_CUDA;
  }
  {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(C_in), 27,
                                static_cast<cuuint64_t>(C_out)};
    const cuuint64_t str[2] = {static_cast<cuuint64_t>(C_in) * 2,
                               static_cast<cuuint64_t>(C_in) * 27 * 2};
    const cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(unstep::conv_weight_box_n(H))};
    if (!encode_bf16(&tmw, w, 3, dims, str, box)) return UNSTEP_ERR_CUDA;
  }
  unstep::ConvParams p{};
  p.y = y;
  p.bias = bias;
  p.dev_error = dev_error;
  p.wait_limit_ns = unstep::kWaitLimitNs;
  p.B = B;
  p.T = T;
  p.H = H;
  p.W = W;
  p.C_in = C_in;
  p.C_out = C_out;
  p.tiles_h = static_cast<int>(tiles_h);
  p.tiles_w = static_cast<int>(tiles_w);
  p.m_tiles = static_cast<int>(m_tiles);
  p.n_tiles = static_cast<int>(n_tiles);
  if (scratch) {
    p.counters = static_cast<unsigned *>(scratch);
    p.slots = reinterpret_cast<float *>(static_cast<char *>(scratch) +
                                        unstep::conv_counter_bytes(sms));
    p.epoch = next_epoch();
  }
  if (unstep::launch_conv3d_causal(tmx, tmw, p, reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  return UNSTEP_OK;
}

size_t unstep_cache_state_bytes(const unstep_cache_t *cache) {
  if (check_shape(cache)) return 0;
  return state_header_bytes(cache) + 2 * unstep_cache_kv_bytes(cache);
}

int unstep_cache_save(const unstep_cache_t *cache, void *host_dst, size_t bytes,
                      unstep_stream_t stream) {
  int rc = check_ready(cache);
  if (rc) return rc;
  if (!host_dst || bytes < unstep_cache_state_bytes(cache)) return UNSTEP_ERR_ARG;
  unsigned char *dst = static_cast<unsigned char *>(host_dst);
  const size_t hb = state_header_bytes(cache), kvb = unstep_cache_kv_bytes(cache);
  std::memset(dst, 0, hb);
  write_state_header(cache, kStateMagic, dst);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(dst + kStateSlotOffset, cache->slot_frame,
                      sizeof(int) * cache->cap_frames, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaMemcpyAsync(dst + hb, cache->k_cache, kvb, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaMemcpyAsync(dst + hb + kvb, cache->v_cache, kvb, cudaMemcpyDeviceToHost, s) !=
          cudaSuccess) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  return UNSTEP_OK;
}

int unstep_cache_restore(unstep_cache_t *cache, const void *host_src, size_t bytes,
                         unstep_stream_t stream) {
  int rc = check_ready(cache);
  if (rc) return rc;
  if (!host_src || bytes < kStateSlotOffset) return UNSTEP_ERR_ARG;
  const unsigned char *src = static_cast<const unsigned char *>(host_src);
  unstep_cache_t saved{};
  rc = read_state_header(src, kStateMagic, &saved);
  if (rc) return rc;
  if (!same_state_shape(cache, &saved)) return UNSTEP_ERR_SHAPE;
  if (bytes < unstep_cache_state_bytes(cache)) return UNSTEP_ERR_ARG;
  // the saved metadata must describe a ring this cache can hold
  if (saved.last_chunk_frames < 0 || saved.last_chunk_frames > cache->cap_frames ||
      saved.frames_written < 0 || saved.frames_written > cache->max_pos_t)
    return UNSTEP_ERR_ARG;
  const size_t hb = state_header_bytes(cache), kvb = unstep_cache_kv_bytes(cache);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(cache->slot_frame, src + kStateSlotOffset,
                      sizeof(int) * cache->cap_frames, cudaMemcpyHostToDevice, s) != cudaSuccess ||
      cudaMemcpyAsync(cache->k_cache, src + hb, kvb, cudaMemcpyHostToDevice, s) != cudaSuccess ||
      cudaMemcpyAsync(cache->v_cache, src + hb + kvb, kvb, cudaMemcpyHostToDevice, s) !=
          cudaSuccess) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  cache->frames_written = saved.frames_written;
  cache->first_frame = saved.first_frame;
  cache->last_chunk_start = saved.last_chunk_start;
  cache->last_chunk_frames = saved.last_chunk_frames;
  return UNSTEP_OK;
}

}  // extern "C"

namespace {

// An initialised 8-bit cache: its base's checks under its own magic, and the scale pointers.
int check_ready_q8(const unstep_q8_cache_t *c) {
  if (!c) return UNSTEP_ERR_ARG;
  int rc = check_shape(&c->base);
  if (rc) return rc;
  if (c->base.initialized != kInitMagicQ8) return UNSTEP_ERR_ARG;
  if (!c->base.k_cache || !c->base.v_cache || !c->base.slot_frame || !c->base.cos_sin ||
      !c->base.dev_error || !c->k_scale || !c->v_scale)
    return UNSTEP_ERR_ARG;
  return UNSTEP_OK;
}

// Ring rows of `count` frames from frame f0 on: at most two ranges.
void ring_rows(const unstep_cache_t *c, int f0, int count, int (&row)[2], int (&len)[2]) {
  const int tf = c->Hg * c->Wg, s0 = f0 % c->cap_frames;
  const int n0 = count < c->cap_frames - s0 ? count : c->cap_frames - s0;
  row[0] = s0 * tf;
  len[0] = n0 * tf;
  row[1] = 0;
  len[1] = (count - n0) * tf;
}

}  // namespace

extern "C" {

size_t unstep_q8_cache_kv_bytes(const unstep_q8_cache_t *cache) {
  return cache ? unstep_cache_kv_bytes(&cache->base) / 2 : 0;
}

size_t unstep_q8_cache_scale_bytes(const unstep_q8_cache_t *cache) {
  return unstep_q8_cache_kv_bytes(cache) / 32;
}

int unstep_q8_cache_init(unstep_q8_cache_t *cache, unstep_stream_t stream) {
  if (!cache) return UNSTEP_ERR_ARG;
  int rc = check_shape(&cache->base);
  if (rc) return rc;
  if (!cache->k_scale || !cache->v_scale) return UNSTEP_ERR_ARG;
  if (!aligned16(cache->k_scale) || !aligned16(cache->v_scale)) return UNSTEP_ERR_ALIGN;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  rc = init_cache(&cache->base, unstep_q8_cache_kv_bytes(cache), kInitMagicQ8, s);
  if (rc) return rc;
  const size_t sb = unstep_q8_cache_scale_bytes(cache);
  if (cudaMemsetAsync(cache->k_scale, 0, sb, s) != cudaSuccess ||
      cudaMemsetAsync(cache->v_scale, 0, sb, s) != cudaSuccess) {
    cudaGetLastError();
    cache->base.initialized = 0;
    return UNSTEP_ERR_CUDA;
  }
  return UNSTEP_OK;
}

int unstep_q8_rope_kv_append(const void *q, void *q_out, const void *k, const void *v,
                             unstep_q8_cache_t *cache, int frame_idx, unstep_grid_t grid,
                             unstep_stream_t stream) {
  int rc = check_ready_q8(cache);
  if (rc) return rc;
  if (!q || !q_out || !k || !v) return UNSTEP_ERR_ARG;
  if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(v))
    return UNSTEP_ERR_ALIGN;
  unstep_cache_t *c = &cache->base;
  const int is_new = unstep_append_plan(c, frame_idx, grid, nullptr);
  if (is_new < 0) return is_new;
  const long long rows = static_cast<long long>(grid.frames) * c->Hg * c->Wg;
  // the kernel numbers the chunk's 8-channel vectors in 31 bits (rows <= 2^30, so nothing overflows)
  if (static_cast<long long>(c->B) * c->H > ((1ll << 31) - 1) / (rows * (c->D / 8)))
    return UNSTEP_ERR_UNSUPPORTED;
  // a thread reads its elements of q, k and v before it writes those of q_out: q_out may be one of
  // them, but not lie across one
  const size_t chunk = act_bytes(c, rows);
  for (const void *in : {q, k, v})
    if (in != q_out && overlap(q_out, chunk, in, chunk)) return UNSTEP_ERR_ARG;
  if (overlaps_rows(q_out, chunk, cache)) return UNSTEP_ERR_ARG;
  unstep::Q8AppendParams p{};
  p.rope = append_params(c, k, v, frame_idx, grid);
  p.rope.q = const_cast<void *>(q);  // read only
  p.rope.rotate_q = 1;
  p.q_out = q_out;
  p.k_scale = static_cast<unsigned char *>(cache->k_scale);
  p.v_scale = static_cast<unsigned char *>(cache->v_scale);
  if (unstep::launch_q8_rope_kv_append(p, reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  note_append(c, frame_idx, grid.frames, is_new == 1);
  return UNSTEP_OK;
}

int unstep_q8_window_attn(const void *q, const unstep_q8_cache_t *cache, int window, void *out,
                          unstep_stream_t stream) {
  const int rc = check_ready_q8(cache);
  if (rc) return rc;
  return window_attn_launch(q, &cache->base, window, out, 0u, false,
                            reinterpret_cast<cudaStream_t>(stream), cache);
}

int unstep_q8_cache_read(const unstep_q8_cache_t *cache, int first_frame, int frames, void *k_out,
                         void *v_out, unstep_stream_t stream) {
  int rc = check_ready_q8(cache);
  if (rc) return rc;
  if ((!k_out && !v_out) || frames < 1) return UNSTEP_ERR_ARG;
  if (!aligned16(k_out) || !aligned16(v_out)) return UNSTEP_ERR_ALIGN;
  const unstep_cache_t *c = &cache->base;
  const long long end = static_cast<long long>(first_frame) + frames;
  if (c->last_chunk_frames < 1 || first_frame < c->first_frame || end > c->frames_written ||
      first_frame < c->frames_written - c->cap_frames)
    return UNSTEP_ERR_WINDOW;
  const size_t out = 2ull * static_cast<size_t>(c->B) * c->H * static_cast<size_t>(frames) * c->Hg *
                     c->Wg * static_cast<size_t>(c->D);
  if (overlap(k_out, out, v_out, out) || overlaps_rows(k_out, out, cache) ||
      overlaps_rows(v_out, out, cache))
    return UNSTEP_ERR_ARG;
  unstep::Q8ReadParams p{};
  p.k_cache = static_cast<const unsigned char *>(c->k_cache);
  p.v_cache = static_cast<const unsigned char *>(c->v_cache);
  p.k_scale = static_cast<const unsigned char *>(cache->k_scale);
  p.v_scale = static_cast<const unsigned char *>(cache->v_scale);
  p.k_out = k_out;
  p.v_out = v_out;
  p.heads = c->B * c->H;
  p.D = c->D;
  p.rows = static_cast<long long>(c->cap_frames) * c->Hg * c->Wg;
  p.n_rows = frames * c->Hg * c->Wg;
  p.dev_error = c->dev_error;
  ring_rows(c, first_frame, frames, p.seg_row, p.seg_len);
  if (unstep::launch_q8_cache_read(p, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  return UNSTEP_OK;
}

size_t unstep_q8_cache_state_bytes(const unstep_q8_cache_t *cache) {
  if (!cache || check_shape(&cache->base)) return 0;
  return state_header_bytes(&cache->base) + 2 * unstep_q8_cache_kv_bytes(cache) +
         2 * unstep_q8_cache_scale_bytes(cache);
}

int unstep_q8_cache_save(const unstep_q8_cache_t *cache, void *host_dst, size_t bytes,
                         unstep_stream_t stream) {
  int rc = check_ready_q8(cache);
  if (rc) return rc;
  if (!host_dst || bytes < unstep_q8_cache_state_bytes(cache)) return UNSTEP_ERR_ARG;
  const unstep_cache_t *c = &cache->base;
  unsigned char *dst = static_cast<unsigned char *>(host_dst);
  const size_t hb = state_header_bytes(c), kvb = unstep_q8_cache_kv_bytes(cache),
               sb = unstep_q8_cache_scale_bytes(cache);
  std::memset(dst, 0, hb);
  write_state_header(c, kStateMagicQ8, dst);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaMemcpyKind down = cudaMemcpyDeviceToHost;
  if (cudaMemcpyAsync(dst + kStateSlotOffset, c->slot_frame, sizeof(int) * c->cap_frames, down,
                      s) != cudaSuccess ||
      cudaMemcpyAsync(dst + hb, c->k_cache, kvb, down, s) != cudaSuccess ||
      cudaMemcpyAsync(dst + hb + kvb, c->v_cache, kvb, down, s) != cudaSuccess ||
      cudaMemcpyAsync(dst + hb + 2 * kvb, cache->k_scale, sb, down, s) != cudaSuccess ||
      cudaMemcpyAsync(dst + hb + 2 * kvb + sb, cache->v_scale, sb, down, s) != cudaSuccess) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  return UNSTEP_OK;
}

int unstep_q8_cache_restore(unstep_q8_cache_t *cache, const void *host_src, size_t bytes,
                            unstep_stream_t stream) {
  int rc = check_ready_q8(cache);
  if (rc) return rc;
  if (!host_src || bytes < kStateSlotOffset) return UNSTEP_ERR_ARG;
  unstep_cache_t *c = &cache->base;
  const unsigned char *src = static_cast<const unsigned char *>(host_src);
  unstep_cache_t saved{};
  rc = read_state_header(src, kStateMagicQ8, &saved);
  if (rc) return rc;
  if (!same_state_shape(c, &saved)) return UNSTEP_ERR_SHAPE;
  if (bytes < unstep_q8_cache_state_bytes(cache)) return UNSTEP_ERR_ARG;
  // the saved metadata must describe a ring this cache can hold: empty, or a latest chunk that
  // ends at the newest frame and does not start before the stream
  const long long chunk_end =
      static_cast<long long>(saved.last_chunk_start) + saved.last_chunk_frames;
  const bool empty = saved.last_chunk_frames == 0 && saved.last_chunk_start == -1 &&
                     saved.frames_written == 0 && saved.first_frame == 0;
  if (!empty && (saved.last_chunk_frames < 1 || saved.last_chunk_frames > c->cap_frames ||
                 saved.first_frame < 0 || saved.last_chunk_start < saved.first_frame ||
                 chunk_end != saved.frames_written || saved.frames_written > c->max_pos_t))
    return UNSTEP_ERR_ARG;
  const size_t hb = state_header_bytes(c), kvb = unstep_q8_cache_kv_bytes(cache),
               sb = unstep_q8_cache_scale_bytes(cache);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaMemcpyKind up = cudaMemcpyHostToDevice;
  if (cudaMemcpyAsync(c->slot_frame, src + kStateSlotOffset, sizeof(int) * c->cap_frames, up,
                      s) != cudaSuccess ||
      cudaMemcpyAsync(c->k_cache, src + hb, kvb, up, s) != cudaSuccess ||
      cudaMemcpyAsync(c->v_cache, src + hb + kvb, kvb, up, s) != cudaSuccess ||
      cudaMemcpyAsync(cache->k_scale, src + hb + 2 * kvb, sb, up, s) != cudaSuccess ||
      cudaMemcpyAsync(cache->v_scale, src + hb + 2 * kvb + sb, sb, up, s) != cudaSuccess) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  c->frames_written = saved.frames_written;
  c->first_frame = saved.first_frame;
  c->last_chunk_start = saved.last_chunk_start;
  c->last_chunk_frames = saved.last_chunk_frames;
  return UNSTEP_OK;
}

}  // extern "C"

namespace {

bool known_type(int t) { return t == UNSTEP_BF16 || t == UNSTEP_F32; }

// A norm's own fields: 0 or an error.
int check_norm(const unstep_norm_t *n, int C) {
  if (n->kind != UNSTEP_NORM_LAYER && n->kind != UNSTEP_NORM_RMS) return UNSTEP_ERR_ARG;
  if (!(n->eps >= 0.f) || !std::isfinite(n->eps) || !known_type(n->param_type))
    return UNSTEP_ERR_ARG;
  if ((n->scale || n->shift) && (n->mod_stride < 0 || (n->mod_stride & 7))) return UNSTEP_ERR_SHAPE;
  if (!aligned16(n->weight) || !aligned16(n->bias) || !aligned16(n->scale) || !aligned16(n->shift))
    return UNSTEP_ERR_ALIGN;
  return C > 0 ? UNSTEP_OK : UNSTEP_ERR_SHAPE;
}

// Sizes that both norm calls share.
int check_rows(long long rows, int C, long long rows_per_group) {
  if (rows < 0 || C < 8 || (C & 7) || rows_per_group < 1) return UNSTEP_ERR_SHAPE;
  if (C > 16384) return UNSTEP_ERR_UNSUPPORTED;
  return UNSTEP_OK;
}

bool bad_stride(long long ld, long long rows, int C) {
  return (ld & 7) || ld < 0 || (rows > 1 && ld < C);
}

// `rows` rows of `bytes` bytes, `stride` bytes apart (none: at is NULL).
struct RowSet {
  uintptr_t at;
  long long rows, stride, bytes;

  RowSet(const void *p, int type, long long ld, long long n, int C)
      : at(reinterpret_cast<uintptr_t>(p)), rows(n), stride(ld * width(type)), bytes(C * width(type)) {
    if (rows > 1 && stride <= bytes) {  // one piece (rows of parameters may even lie on each other)
      bytes += (rows - 1) * stride;
      rows = 1;
    }
  }
  static long long width(int type) { return type == UNSTEP_F32 ? 4 : 2; }
  uintptr_t end() const { return at + static_cast<uintptr_t>((rows - 1) * stride + bytes); }
};

// Whether row i of a shares a byte with a row of b.
bool row_meets(const RowSet &a, long long i, const RowSet &b) {
  const long long d = static_cast<long long>(a.at - b.at) + i * a.stride;  // from b's first row
  if (d + a.bytes <= 0) return false;
  if (b.rows == 1) return d < b.bytes;
  const long long j = d < b.bytes ? 0 : (d - b.bytes) / b.stride + 1;  // b's first row to end after d
  return j < b.rows && j * b.stride < d + a.bytes;
}

// Whether two sets share a byte.  Sets of one stride (column blocks of a wider tensor) share one
// where the first row of either is in it: a meeting pair of later rows moves back to one.
bool share(const RowSet &a, const RowSet &b) {
  if (!a.at || !b.at || a.end() <= b.at || b.end() <= a.at) return false;
  if (a.rows > b.rows) return share(b, a);
  if (row_meets(a, 0, b) || row_meets(b, 0, a)) return true;
  if (a.rows > 1 && a.stride == b.stride) return false;
  for (long long i = 1; i < a.rows; ++i)
    if (row_meets(a, i, b)) return true;
  return false;
}

// Whether an output shares a byte with a norm's parameters for `groups` groups.
bool shares_parameters(const RowSet &out, const unstep_norm_t &n, long long groups, int C) {
  const int t = n.param_type;
  return share(out, {n.weight, t, 0, 1, C}) || share(out, {n.bias, t, 0, 1, C}) ||
         share(out, {n.scale, t, n.mod_stride, groups, C}) ||
         share(out, {n.shift, t, n.mod_stride, groups, C});
}

}  // namespace

extern "C" {

int unstep_norm_modulate(const void *x, int x_type, long long ldx, void *y, long long ldy,
                         long long rows, int C, long long rows_per_group,
                         const unstep_norm_t *norm, unstep_stream_t stream) {
  if (!norm || !known_type(x_type)) return UNSTEP_ERR_ARG;
  int rc = check_rows(rows, C, rows_per_group);
  if (rc) return rc;
  rc = check_norm(norm, C);
  if (rc) return rc;
  if (rows == 0) return UNSTEP_OK;
  if (!x || !y) return UNSTEP_ERR_ARG;
  if (bad_stride(ldx, rows, C) || bad_stride(ldy, rows, C)) return UNSTEP_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(y)) return UNSTEP_ERR_ALIGN;
  // the rows run in no order, and one is loaded while the one before it is stored
  const long long groups = (rows - 1) / rows_per_group + 1;
  const RowSet out(y, UNSTEP_BF16, ldy, rows, C);
  const bool onto_x = y == x && x_type == UNSTEP_BF16 && ldy == ldx;
  if ((!onto_x && (y == x || share(out, {x, x_type, ldx, rows, C}))) ||
      shares_parameters(out, *norm, groups, C))
    return UNSTEP_ERR_ARG;
  unstep::NormParams p{};
  p.x = x;
  p.x_type = x_type;
  p.ldx = ldx;
  p.h = y;
  p.ldh = ldy;
  p.rows = rows;
  p.C = C;
  p.rows_per_group = rows_per_group;
  p.next = *norm;
  if (unstep::launch_block_norm(p, false, reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  return UNSTEP_OK;
}

int unstep_gate_residual_norm(const void *x, int x_type, long long ldx, const void *y,
                              long long ldy, const void *gate, int gate_type,
                              long long gate_stride, float res_scale, const unstep_norm_t *post,
                              const unstep_norm_t *next, void *x_out, long long ldxo, void *h,
                              long long ldh, long long rows, int C, long long rows_per_group,
                              unstep_stream_t stream) {
  if (!known_type(x_type) || !known_type(gate_type) || !std::isfinite(res_scale))
    return UNSTEP_ERR_ARG;
  if ((next == nullptr) != (h == nullptr) && rows > 0) return UNSTEP_ERR_ARG;
  int rc = check_rows(rows, C, rows_per_group);
  if (rc) return rc;
  if (post && (rc = check_norm(post, C))) return rc;
  if (next && (rc = check_norm(next, C))) return rc;
  if (rows == 0) return UNSTEP_OK;
  if (!x || !y || !x_out) return UNSTEP_ERR_ARG;
  if (bad_stride(ldx, rows, C) || bad_stride(ldy, rows, C) || bad_stride(ldxo, rows, C) ||
      (h && bad_stride(ldh, rows, C)) || (gate && (gate_stride < 0 || (gate_stride & 7))))
    return UNSTEP_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(y) || !aligned16(gate) || !aligned16(x_out) || !aligned16(h))
    return UNSTEP_ERR_ALIGN;
  const long long groups = (rows - 1) / rows_per_group + 1;
  const RowSet x_set(x, x_type, ldx, rows, C), y_set(y, UNSTEP_BF16, ldy, rows, C);
  const RowSet sum_set(x_out, x_type, ldxo, rows, C), h_set(h, UNSTEP_BF16, ldh, rows, C);
  if ((x_out == x ? ldxo != ldx : share(sum_set, x_set)) || share(h_set, x_set) ||
      share(h_set, sum_set))
    return UNSTEP_ERR_ARG;
  for (const RowSet *out : {&sum_set, &h_set})
    if (share(*out, y_set) || share(*out, {gate, gate_type, gate_stride, groups, C}) ||
        (post && shares_parameters(*out, *post, groups, C)) ||
        (next && shares_parameters(*out, *next, groups, C)))
      return UNSTEP_ERR_ARG;
  unstep::NormParams p{};
  p.x = x;
  p.x_type = x_type;
  p.ldx = ldx;
  p.y = y;
  p.ldy = ldy;
  p.gate = gate;
  p.gate_type = gate_type;
  p.gate_stride = gate_stride;
  p.res_scale = res_scale;
  p.x_out = x_out;
  p.ldxo = ldxo;
  p.h = h;
  p.ldh = ldh;
  p.rows = rows;
  p.C = C;
  p.rows_per_group = rows_per_group;
  p.has_post = post ? 1 : 0;
  if (post) p.post = *post;
  if (next) p.next = *next;
  if (unstep::launch_block_norm(p, true, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  return UNSTEP_OK;
}

int unstep_get_device_error(const unstep_cache_t *cache, unstep_stream_t stream) {
  if (!cache || !cache->dev_error) return UNSTEP_ERR_ARG;
  int v = 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(&v, cache->dev_error, sizeof(int), cudaMemcpyDeviceToHost, s) !=
          cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  return v;
}

int unstep_selftest_wait_timeout(int *dev_error, uint64_t limit_ns, unstep_stream_t stream) {
  if (!dev_error) return UNSTEP_ERR_ARG;
  if (unstep::launch_wait_timeout_selftest(dev_error, limit_ns,
                                           reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  return UNSTEP_OK;
}

int unstep_selftest_exp2(const float *x, float *y_poly, float *y_mufu, int n,
                         unstep_stream_t stream) {
  if (!x || !y_poly || !y_mufu || n < 0) return UNSTEP_ERR_ARG;
  if (n == 0) return UNSTEP_OK;
  if (unstep::launch_exp2_selftest(x, y_poly, y_mufu, n, reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess) {
    cudaGetLastError();
    return UNSTEP_ERR_CUDA;
  }
  return UNSTEP_OK;
}

}  // extern "C"
