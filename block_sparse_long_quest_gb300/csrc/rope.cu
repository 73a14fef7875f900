// rope.cu — rotary positions of query and key rows (kt_apply_rope).
//
// A warp takes the head rows of one token (or a slice of them, for short calls):
// it computes the token's 64 (cos, sin) once, holds a lane's eight in registers and
// streams the heads through, four rows at a time, 8 lanes a row, two 16-byte
// vectors a lane.  Bound by HBM: each row is read once and written once as
// binary16.
#include <cstring>

#include "rope.cuh"

namespace kt {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;

struct Params {
  kt_rope rope;
  const int32_t* positions;  // nullable: then from cu and seq_lens
  const int32_t* cu;
  const int32_t* seq_lens;
  const void* q;
  const void* k;
  long long qs, ks;
  __half* q_out;
  __half* k_out;
  int hq, hk, tokens, heads_per, B;
};

// Two groups of four rows in flight a warp (NB 2, at most 80 registers, 24 warps an
// SM): 8192 tokens of 32 + 8 bf16 heads take 29.9 us, 83% of the measured copy
// rate; 5003 of 16 + 4 binary32 heads 15.4 us, 74% (626 CTAs at three an SM: a wave
// and four tenths).  When the phases still came from the parameters, NB 2 took 31.1,
// one group at 64 registers 32.1, two at 128 registers 34.6 and at 64 34.2.
template <class T, int M>
__global__ void __launch_bounds__(THREADS, 3) rope_kernel(const __grid_constant__ Params p) {
  __shared__ __align__(16) float2 cs[WARPS][64];
  __shared__ RopeShared rs;
  if (M != ROPE_M_NONE) {
    rope_prepare(p.rope, rs, threadIdx.x, THREADS);
    __syncthreads();
  }
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = (int)blockIdx.x * WARPS + warp;
  if (t >= p.tokens) return;
  if (p.cu && (t < p.cu[0] || t >= p.cu[p.B])) return;  // rows of no sequence
  const int h0 = (int)blockIdx.y * p.heads_per, h1 = min(h0 + p.heads_per, p.hq + p.hk);
  int pos = 0;
  if (p.positions) {
    pos = p.positions[t];
  } else if (M != ROPE_M_NONE) {
    const int s = row_sequence(p.cu, p.B, t, lane);
    pos = p.seq_lens[s] + (t - p.cu[s]);
  }
  rope_token<M, 2>(p.rope, rs, cs[warp], pos, t, h0, h1, static_cast<const T*>(p.q), p.qs, p.hq,
                   p.q_out, static_cast<const T*>(p.k), p.ks, p.hk, p.k_out, lane);
}

template <class T>
cudaError_t launch_mode(const cudaLaunchConfig_t& cfg, int mode, const Params& p) {
  switch (mode) {
    case ROPE_M_NONE: return cudaLaunchKernelEx(&cfg, rope_kernel<T, ROPE_M_NONE>, p);
    case ROPE_M_VECTORS: return cudaLaunchKernelEx(&cfg, rope_kernel<T, ROPE_M_VECTORS>, p);
    case ROPE_M_PAIRS: return cudaLaunchKernelEx(&cfg, rope_kernel<T, ROPE_M_PAIRS>, p);
    case ROPE_M_ANY: return cudaLaunchKernelEx(&cfg, rope_kernel<T, ROPE_M_ANY>, p);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch& a, cudaStream_t stream) {
  if (a.tokens <= 0 || a.hq + a.hk <= 0) return cudaSuccess;
  Params p;
  std::memset(&p, 0, sizeof(p));
  if (a.rope) p.rope = *a.rope;
  p.cu = a.cu;
  p.seq_lens = a.seq_lens;
  p.B = a.B;
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
  // one warp a token where that gives every SM 16 warps; else the heads are sliced
  const int H = a.hq + a.hk;
  p.heads_per = H;
  while (p.heads_per > 4 &&
         (long long)a.tokens * ((H + p.heads_per - 1) / p.heads_per) < 16ll * a.num_sms)
    p.heads_per = (((p.heads_per + 1) / 2) + 3) & ~3;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)a.tokens + WARPS - 1) / WARPS),
                     (unsigned)((H + p.heads_per - 1) / p.heads_per));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;

  const int mode = rope_mode(a.rope);
  switch (a.dtype) {
    case KT_F16: return launch_mode<__half>(cfg, mode, p);
    case KT_BF16: return launch_mode<__nv_bfloat16>(cfg, mode, p);
    case KT_F32: return launch_mode<float>(cfg, mode, p);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kt
