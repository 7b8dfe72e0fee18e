// Attention over the 8-bit paged key/value cache (np_kv_attend).
//
// One warp per (new token, query head): lane l holds D/32 neighbouring
// elements of q and of the output, and the warp walks the visible keys one
// after another with a running maximum and sum, all in fp32:
//   s_j = (q . k_j) * k_scale * scale,  m' = max(m, s_j),
//   l' = l 2^(m - m') + 2^(s_j - m'),  o' = o 2^(m - m') + 2^(s_j - m') v_j.
#include "np_kv.cuh"

namespace np {

namespace {

template <typename T, int D>
__global__ void __launch_bounds__(128) attend_simple_kernel(const KvAttend a) {
  constexpr int E = D / 32;
  const int warp = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int tok = warp / a.Hq, h = warp % a.Hq;
  if (tok >= a.batch.n_tokens) return;
  KvSeq s{};
  bool found = false;
  for (int i = 0; i < a.batch.n_seqs; ++i) {
    const KvSeq t = kv_seq(a.kv, a.batch, i);
    if (tok >= t.begin && tok < t.begin + t.n) {
      s = t;
      found = true;
    }
  }
  if (!found) return;
  const int pos = s.len - s.n + tok - s.begin;
  const int kvh = h / (a.Hq / a.kv.H);
  const T* q = static_cast<const T*>(a.q) + tok * a.q_tok + h * a.q_head + lane * E;
  float qv[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    qv[i] = kv_to_float<T>(q[i]);
    o[i] = 0.f;
  }
  for (int j = 0; j <= pos; ++j) {
    if (a.window > 0 && j <= pos - a.window && j >= a.sinks) {
      j = pos - a.window;
      continue;
    }
    const int page = a.kv.table[(size_t)s.row * a.kv.max_pages + j / kKvPage];
    if (page < 0 || page >= a.kv.n_pages) {
      if (page != -1) atomicExch(a.kv.err, kDevErrBounds);
      continue;
    }
    const size_t block = (size_t)page * a.kv.H + kvh;
    const uint8_t* k = a.kv.k + (block * kKvPage + j % kKvPage) * D + lane * E;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) x = fmaf(qv[i], f16x2_to_f32x2(e4m3x2_to_f16x2(k[i])).x, x);
    x = warp_sum(x) * a.kv.k_scale[block] * a.scale_log2;
    const float mn = fmaxf(m, x), ref = mn == -INFINITY ? 0.f : mn;
    const float c = exp2f(m - ref), p = exp2f(x - ref);
    const float pv = p * a.kv.v_scale[block];
    const uint8_t* v = a.kv.v + (block * D + lane * E) * kKvPage + j % kKvPage;
    l = l * c + p;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = fmaf(pv, f16x2_to_f32x2(e4m3x2_to_f16x2(v[i * kKvPage])).x, o[i] * c);
    m = mn;
  }
  T* out = static_cast<T*>(a.out) + tok * a.o_tok + h * a.o_head + lane * E;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < E; ++i) out[i] = kv_from_float<T>(o[i] * inv);
}

template <typename T>
cudaError_t launch_typed(const KvAttend& a, cudaStream_t st) {
  const long long warps = (long long)a.batch.n_tokens * a.Hq;
  const unsigned grid = (unsigned)((warps + 3) / 4);
  switch (a.kv.D) {
    case 64: attend_simple_kernel<T, 64><<<grid, 128, 0, st>>>(a); break;
    case 128: attend_simple_kernel<T, 128><<<grid, 128, 0, st>>>(a); break;
    case 256: attend_simple_kernel<T, 256><<<grid, 128, 0, st>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace

size_t kv_attend_workspace(int) { return 16; }

cudaError_t launch_kv_attend(const KvAttend& a, cudaStream_t st) {
  switch (a.dtype) {
    case 0: return launch_typed<float>(a, st);
    case 1: return launch_typed<__half>(a, st);
    default: return launch_typed<__nv_bfloat16>(a, st);
  }
}

}  // namespace np
