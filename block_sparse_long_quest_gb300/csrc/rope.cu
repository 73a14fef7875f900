// rope.cu — rotary positions of query and key rows (kt_apply_rope).
//
// A CTA takes a few tokens: it computes their (cos, sin) once into shared
// memory (rope.cuh) and then streams all heads of those tokens through, 8
// lanes a head row, two 16-byte vectors a lane.  Bound by HBM: each row is read
// once and written once as binary16.
#include "rope.cuh"

namespace kt {
namespace {

constexpr int THREADS = 256;
constexpr int MAX_TOK = 4;  // tokens of a CTA

struct Params {
  kt_rope rope;
  const int32_t* positions;
  const void* q;
  const void* k;
  long long qs, ks;
  __half* q_out;
  __half* k_out;
  int hq, hk, tokens, per_cta;
};

template <class T>
__global__ void __launch_bounds__(THREADS) rope_kernel(const __grid_constant__ Params p) {
  __shared__ __align__(16) float2 cs[MAX_TOK * 64];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  const int t0 = (int)blockIdx.x * p.per_cta, ntok = min(p.per_cta, p.tokens - t0);
  for (int i = tid; i < ntok * 64; i += THREADS)
    if ((i & 63) < p.rope.rotary_dim / 2)
      cs[i] = rope_cos_sin(p.rope, i & 63, p.positions[t0 + (i >> 6)]);
  __syncthreads();
  rope_tokens(p.rope, cs, t0, ntok, static_cast<const T*>(p.q), p.qs, p.hq, p.q_out,
              static_cast<const T*>(p.k), p.ks, p.hk, p.k_out, tid, THREADS);
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch& a, cudaStream_t stream) {
  if (a.tokens <= 0 || a.hq + a.hk <= 0) return cudaSuccess;
  Params p;
  p.rope = *a.rope;
  p.positions = a.positions;
  p.q = a.q;
  p.k = a.k;
  p.qs = a.qs;
  p.ks = a.ks;
  p.q_out = a.q_out;
  p.k_out = a.k_out;
  p.hq = a.hq;
  p.hk = a.hk;
  p.tokens = a.tokens;
  p.per_cta = a.tokens >= 4 * a.num_sms ? MAX_TOK : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)a.tokens + p.per_cta - 1) / p.per_cta));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  switch (a.dtype) {
    case KT_F16: return cudaLaunchKernelEx(&cfg, rope_kernel<__half>, p);
    case KT_BF16: return cudaLaunchKernelEx(&cfg, rope_kernel<__nv_bfloat16>, p);
    case KT_F32: return cudaLaunchKernelEx(&cfg, rope_kernel<float>, p);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kt
