// sa_api_serving.cu -- C ABI of the serving-step operators: rotary positions,
// the page write and read-back, and the packed prefill.  Host-side argument
// checks and launches; nothing here allocates, frees or synchronises.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/sa.h"
#include "serving.h"
#include "strided.h"

namespace {

bool rope_ok(const sa_rope* r) {
  return r->rotary_dim >= 2 && r->rotary_dim <= 2 * SA_ROPE_MAX_PAIRS && r->rotary_dim % 2 == 0 &&
         r->reserved_ == 0 && std::isfinite(r->mscale);
}

}  // namespace

namespace sa {

constexpr int kMaxDevices = 64;

int sm_count() {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 152;
  if (dev < kMaxDevices && known[dev].load(std::memory_order_relaxed) > 0)
    return known[dev].load(std::memory_order_relaxed);
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 152;
  if (dev < kMaxDevices) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

bool allow_smem(const void* kernel, int bytes) {
  constexpr int kSlots = 256;  // (kernel, device) pairs seen, open addressing
  static std::atomic<uintptr_t> seen[kSlots];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return false;
  const uintptr_t key = reinterpret_cast<uintptr_t>(kernel) * kMaxDevices + static_cast<uintptr_t>(dev);
  const unsigned h = static_cast<unsigned>((key * 0x9E3779B97F4A7C15ull) >> 56);
  for (int i = 0; i < kSlots; ++i) {
    const uintptr_t at = seen[(h + i) % kSlots].load(std::memory_order_acquire);
    if (at == key) return true;
    if (at == 0) break;
  }
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  for (int i = 0; i < kSlots; ++i) {
    uintptr_t none = 0;
    if (seen[(h + i) % kSlots].compare_exchange_strong(none, key, std::memory_order_acq_rel) || none == key) break;
  }
  return true;
}

}  // namespace sa

extern "C" {

int sa_rope_table(const sa_rope_config* c, sa_rope* out) {
  if (!c || !out) return SA_ERR_NULL;
  if (c->scaling < SA_ROPE_NONE || c->scaling > SA_ROPE_FREQS) return SA_ERR_UNSUPPORTED;
  const int R = c->rotary_dim;
  if (R < 2 || R > 2 * SA_ROPE_MAX_PAIRS || R % 2) return SA_ERR_SHAPE;
  if (!std::isfinite(c->mscale)) return SA_ERR_SHAPE;
  if (c->scaling == SA_ROPE_FREQS) {
    if (!c->inv_freq) return SA_ERR_NULL;
  } else if (!(c->base > 0.0) || !std::isfinite(c->base)) {
    return SA_ERR_SHAPE;
  }
  const bool scaled = c->scaling == SA_ROPE_LINEAR || c->scaling == SA_ROPE_NTK || c->scaling == SA_ROPE_RAMP;
  if (scaled && (!(c->factor > 0.0) || !std::isfinite(c->factor))) return SA_ERR_SHAPE;
  if (c->scaling == SA_ROPE_NTK && R == 2) return SA_ERR_SHAPE;
  if (c->scaling == SA_ROPE_RAMP &&
      (!(c->original_len > 0.0) || !std::isfinite(c->original_len) || !(c->ramp_high > c->ramp_low) ||
       !std::isfinite(c->ramp_low) || !std::isfinite(c->ramp_high)))
    return SA_ERR_SHAPE;
  sa_rope r;
  memset(&r, 0, sizeof(r));
  r.rotary_dim = R;
  r.interleaved = c->interleaved ? 1 : 0;
  r.mscale = c->mscale == 0.f ? 1.f : c->mscale;
  const double two_pi = 6.283185307179586476925286766559;
  double base = c->base;
  if (c->scaling == SA_ROPE_NTK) base *= std::pow(c->factor, static_cast<double>(R) / (R - 2));
  for (int i = 0; i < R / 2; ++i) {
    double f = c->scaling == SA_ROPE_FREQS ? c->inv_freq[i] : std::pow(base, -2.0 * i / R);
    if (c->scaling == SA_ROPE_LINEAR) f /= c->factor;
    if (c->scaling == SA_ROPE_RAMP) {
      double g = (c->original_len * f / two_pi - c->ramp_low) / (c->ramp_high - c->ramp_low);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      f = f * g + f / c->factor * (1.0 - g);
    }
    if (!std::isfinite(f)) return SA_ERR_SHAPE;
    // the turn's fraction as 64 bits (a whole turn per position changes nothing)
    double turns = f / two_pi;
    turns -= std::floor(turns);
    r.turns[i] = turns >= 1.0 ? 0 : static_cast<uint64_t>(std::ldexp(turns, 64));
  }
  *out = r;
  return SA_OK;
}

int rotary_embed(const sa_rotary_params* p, void* stream) {
  if (!p || !p->q || !p->q_out || !p->positions || !p->rope) return SA_ERR_NULL;
  if ((p->k == nullptr) != (p->k_out == nullptr)) return SA_ERR_NULL;
  const size_t es = dtype_bytes(p->dtype);
  if (es == 0) return SA_ERR_DTYPE;
  if (p->B <= 0 || p->S < 0 || p->Hq <= 0 || p->D <= 0 || (p->k && p->Hk <= 0) || p->pos_stride < 0)
    return SA_ERR_SHAPE;
  if (!rope_ok(p->rope) || p->rope->rotary_dim > p->D) return SA_ERR_SHAPE;
  if (p->B >= kMaxInt || p->S >= kMaxInt || p->B * p->S >= kMaxTokens || p->Hq >= kMaxInt / 4 ||
      p->Hk >= kMaxInt / 4 || p->D - p->rope->rotary_dim / 2 > 256)
    return SA_ERR_UNSUPPORTED;
  auto tensor = [&](const void* ptr, int64_t H, const int64_t (&st)[3]) {
    return Strided{ptr, es, 3, {p->B, p->S, H}, {st[0], st[1], st[2]}, p->D};
  };
  const Strided x[2] = {tensor(p->q, p->Hq, p->q_strides), tensor(p->k, p->Hk, p->k_strides)};
  const Strided y[2] = {tensor(p->q_out, p->Hq, p->q_out_strides), tensor(p->k_out, p->Hk, p->k_out_strides)};
  const int n = p->k ? 2 : 1;
  if (!aligned(p->positions, p->pos_is_i64 ? 8 : 4)) return SA_ERR_ALIGN;
  for (int i = 0; i < n; ++i) {
    if (!x[i].strides_ok() || !y[i].strides_ok() || !y[i].distinct()) return SA_ERR_SHAPE;
    if (!aligned(x[i].p, es) || !aligned(y[i].p, es)) return SA_ERR_ALIGN;
  }
  if (p->S == 0) return SA_OK;
  const size_t pos_bytes = static_cast<size_t>((p->B - 1) * p->pos_stride + p->S) * (p->pos_is_i64 ? 8 : 4);
  for (int i = 0; i < n; ++i) {
    for (int j = 0; j < n; ++j)
      if (!(i == j && same(x[j], y[i])) && overlap(x[j], y[i])) return SA_ERR_OVERLAP;
    if (ranges_meet(y[i].p, y[i].extent(), p->positions, pos_bytes)) return SA_ERR_OVERLAP;
  }
  if (n == 2 && overlap(y[0], y[1])) return SA_ERR_OVERLAP;
  sa::RotaryArgs a;
  memset(&a, 0, sizeof(a));
  const int R = p->rope->rotary_dim;
  a.vec = p->D % 16 == 0 && R % 16 == 0;
  for (int i = 0; i < n; ++i) {
    a.x[i] = x[i].p;
    a.y[i] = const_cast<void*>(y[i].p);
    a.H[i] = static_cast<int>(i ? p->Hk : p->Hq);
    a.in_place[i] = same(x[i], y[i]);
    a.vec = a.vec && x[i].vec16() && y[i].vec16();
    for (int k = 0; k < 3; ++k) {
      a.xs[i][k] = x[i].n[k] > 1 ? x[i].st[k] : 0;
      a.ys[i][k] = y[i].n[k] > 1 ? y[i].st[k] : 0;
    }
  }
  a.positions = p->positions;
  a.pos_is_i64 = p->pos_is_i64 ? 1 : 0;
  a.pos_stride = p->pos_stride;
  a.S = static_cast<int>(p->S);
  a.T = static_cast<int>(p->B * p->S);
  a.D = static_cast<int>(p->D);
  a.rope = *p->rope;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  sa::mark_event(sa::kernel_event_before(), st);
  const int rc = sa::launch_rotary(a, p->dtype, st);
  sa::mark_event(sa::kernel_event_after(), st);
  return rc == 0 ? SA_OK : SA_ERR_LAUNCH;
}

// Checks shared by the page write and read-back; fills the kernel's arguments.
static int kv_pages_args(const sa_kv_pages_params* p, bool write, sa::KvPagesArgs& a) {
  if (!p || !p->k || !p->v || !p->k_pool || !p->v_pool || !p->block_table || !p->ctx_len)
    return SA_ERR_NULL;
  const size_t es = dtype_bytes(p->dtype);
  const bool fp8 = p->pool_format == SA_FP8_E4M3_PAGE;
  if (es == 0 || (p->pool_format != 0 && !fp8)) return SA_ERR_DTYPE;
  if (p->T < 0 || p->B <= 0 || p->Hkv <= 0 || p->D <= 0 || p->page_tokens <= 0 || p->max_pages <= 0 ||
      p->num_pages <= 0)
    return SA_ERR_SHAPE;
  if (!p->seq_start && p->T != p->B) return SA_ERR_SHAPE;
  if (p->rope && (!rope_ok(p->rope) || p->rope->rotary_dim > p->D)) return SA_ERR_SHAPE;
  if (p->rope && !write) return SA_ERR_UNSUPPORTED;
  if (p->D > 1024 || p->T >= kMaxTokens || p->B >= kMaxInt || p->Hkv >= (int64_t(1) << 20) ||
      p->page_tokens >= kMaxInt || p->max_pages >= kMaxInt || p->num_pages >= kMaxInt ||
      p->max_pages * p->page_tokens >= kMaxInt)
    return SA_ERR_UNSUPPORTED;
  if (fp8 && (!(p->D == 64 || p->D == 128 || p->D == 256) || p->page_tokens % 16 != 0))
    return SA_ERR_UNSUPPORTED;
  if (fp8 ? !(aligned(p->k_pool, 16) && aligned(p->v_pool, 16))
          : !(aligned(p->k_pool, es) && aligned(p->v_pool, es)))
    return SA_ERR_ALIGN;
  const Strided x[2] = {{p->k, es, 2, {p->T, p->Hkv, 1}, {p->k_strides[0], p->k_strides[1], 0}, p->D},
                        {p->v, es, 2, {p->T, p->Hkv, 1}, {p->v_strides[0], p->v_strides[1], 0}, p->D}};
  for (int i = 0; i < 2; ++i) {
    if (!x[i].strides_ok() || (!write && !x[i].distinct())) return SA_ERR_SHAPE;
    if (!aligned(x[i].p, es)) return SA_ERR_ALIGN;
  }
  const size_t row = fp8 ? static_cast<size_t>(p->D + 1) : static_cast<size_t>(p->D) * es;
  const int64_t head_page = p->page_tokens * static_cast<int64_t>(row);  // (below 2^43)
  if (p->num_pages * p->Hkv > (int64_t(1) << 62) / head_page) return SA_ERR_UNSUPPORTED;
  const size_t pool = static_cast<size_t>(p->num_pages * p->Hkv * head_page);
  if (ranges_meet(p->k_pool, pool, p->v_pool, pool)) return SA_ERR_OVERLAP;
  if (p->T > 0) {
    for (int i = 0; i < 2; ++i)
      if (ranges_meet(x[i].p, x[i].extent(), p->k_pool, pool) || ranges_meet(x[i].p, x[i].extent(), p->v_pool, pool))
        return SA_ERR_OVERLAP;
    if (!write && overlap(x[0], x[1])) return SA_ERR_OVERLAP;
  }
  memset(&a, 0, sizeof(a));
  a.pool[0] = p->k_pool;
  a.pool[1] = p->v_pool;
  a.aligned = 1;
  for (int i = 0; i < 2; ++i) {
    a.x[i] = const_cast<void*>(x[i].p);
    a.xs[i][0] = x[i].st[0];
    a.xs[i][1] = x[i].st[1];
    a.aligned = a.aligned && x[i].vec16() && p->D * static_cast<int64_t>(es) % 16 == 0 &&
                (fp8 || aligned(a.pool[i], 16));
  }
  a.block_table = p->block_table;
  a.ctx_len = p->ctx_len;
  a.seq_start = p->seq_start;
  a.err_word = p->err_word;
  a.fp8 = fp8;
  a.has_rope = p->rope != nullptr;
  if (p->rope) a.rope = *p->rope;
  a.T = static_cast<int>(p->T);
  a.B = static_cast<int>(p->B);
  a.Hkv = static_cast<int>(p->Hkv);
  a.D = static_cast<int>(p->D);
  a.page_tokens = p->page_tokens;
  a.max_pages = p->max_pages;
  a.num_pages = p->num_pages;
  return SA_OK;
}

int paged_kv_write(const sa_kv_pages_params* p, void* stream) {
  sa::KvPagesArgs a;
  const int rc = kv_pages_args(p, true, a);
  if (rc != SA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  sa::mark_event(sa::kernel_event_before(), st);
  const int lrc = sa::launch_kv_write(a, p->dtype, st);
  sa::mark_event(sa::kernel_event_after(), st);
  return lrc == 0 ? SA_OK : SA_ERR_LAUNCH;
}

int paged_kv_read(const sa_kv_pages_params* p, void* stream) {
  sa::KvPagesArgs a;
  const int rc = kv_pages_args(p, false, a);
  if (rc != SA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  sa::mark_event(sa::kernel_event_before(), st);
  const int lrc = sa::launch_kv_read(a, p->dtype, st);
  sa::mark_event(sa::kernel_event_after(), st);
  return lrc == 0 ? SA_OK : SA_ERR_LAUNCH;
}

int attn_prefill_packed(const sa_packed_params* p, void* stream) {
  if (!p || !p->q || !p->k || !p->v || !p->y || !p->q_start) return SA_ERR_NULL;
  const size_t es = dtype_bytes(p->dtype);
  if (es == 0) return SA_ERR_DTYPE;
  if (p->B <= 0 || p->Tq < 0 || p->Tk < 0 || p->Hq <= 0 || p->Hkv <= 0 || p->D <= 0 || p->Hq % p->Hkv != 0)
    return SA_ERR_SHAPE;
  if (!p->k_start && p->Tq != p->Tk) return SA_ERR_SHAPE;
  if (!std::isfinite(p->scale) || !std::isfinite(p->softcap) || p->softcap < 0.f) return SA_ERR_SHAPE;
  if (p->D > 256 || p->D % 4 != 0 || p->Tq >= (int64_t(1) << 30) || p->Tk >= (int64_t(1) << 30) ||
      p->B >= (int64_t(1) << 24) || p->Hq > 65535)
    return SA_ERR_UNSUPPORTED;
  auto tensor = [&](const void* ptr, int64_t T, int64_t H, const int64_t (&st)[2]) {
    return Strided{ptr, es, 2, {T, H, 1}, {st[0], st[1], 0}, p->D};
  };
  const Strided q = tensor(p->q, p->Tq, p->Hq, p->q_strides), y = tensor(p->y, p->Tq, p->Hq, p->y_strides);
  const Strided k = tensor(p->k, p->Tk, p->Hkv, p->k_strides), v = tensor(p->v, p->Tk, p->Hkv, p->v_strides);
  const Strided* all[4] = {&q, &k, &v, &y};
  for (const Strided* t : all) {
    if (!t->strides_ok()) return SA_ERR_SHAPE;
    if (!aligned(t->p, es)) return SA_ERR_ALIGN;
  }
  if (!y.distinct()) return SA_ERR_SHAPE;
  if (overlap(q, y) || overlap(k, y) || overlap(v, y)) return SA_ERR_OVERLAP;
  if (p->Tq == 0) return SA_OK;
  sa::PackedArgs a;
  memset(&a, 0, sizeof(a));
  a.q = p->q;
  a.k = p->k;
  a.v = p->v;
  a.y = p->y;
  a.q_start = p->q_start;
  a.k_start = p->k_start ? p->k_start : p->q_start;
  a.err_word = p->err_word;
  a.dtype = p->dtype;
  a.causal = p->causal ? 1 : 0;
  a.B = p->B;
  a.Tq = p->Tq;
  a.Tk = p->Tk;
  a.Hq = p->Hq;
  a.Hkv = p->Hkv;
  a.D = p->D;
  for (int i = 0; i < 2; ++i) {
    a.qs[i] = q.st[i];
    a.ks[i] = k.st[i];
    a.vs[i] = v.st[i];
    a.ys[i] = y.st[i];
  }
  a.scale = p->scale != 0.f ? p->scale : 1.0f / sqrtf(static_cast<float>(p->D));
  a.softcap = p->softcap;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  bool vec = true;  // 16-byte rows whose strides a tensor map can hold
  for (const Strided* t : all) {
    vec = vec && t->vec16();
    for (int i = 0; i < 2; ++i) vec = vec && (t->n[i] <= 1 || t->st[i] > 0);
  }
  sa::mark_event(sa::kernel_event_before(), st);
  const int rc = vec && sa::packed_tc_supported(a) ? sa::launch_packed_tc(a, st) : sa::launch_packed_simt(a, st);
  sa::mark_event(sa::kernel_event_after(), st);
  return rc == 0 ? SA_OK : SA_ERR_LAUNCH;
}

}  // extern "C"
