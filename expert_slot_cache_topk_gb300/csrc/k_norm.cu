// Norms around a block, fused with its gate and residual scale, per token:
//   n  = b * rsqrt(mean(b^2) + eps) * post_w
//   x' = x + res_scale * gate * n
//   y  = x' * rsqrt(mean(x'^2) + eps) * pre_w
// One block of threads per row (rows b, b + grid, ...): x, b and the gate are
// read once into registers, the two means are block sums of f32 squares, and
// x' feeds the second norm before it is rounded.  The bound is memory: x and b
// read, x' and y written (the weights stay in registers from row to row).
#include "attn_common.cuh"

namespace moe {
namespace {

using namespace attn;

struct NormArgs {
  const void *x, *block, *post, *gate, *pre;
  void *x_out, *y;
  long long tokens, x_row, block_row, gate_row, x_out_row, y_row;
  int hidden, gate_col;
  float res_scale, eps;
};

// Sum over the block; `red` alternates between calls, so one barrier is enough:
// a buffer is written again only after the barrier of the call in between,
// which no thread passes before it has read this one.
__device__ __forceinline__ float block_add(float v, float* red, int warps) {
  v = warp_add(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < warps; ++w) s += red[w];
  return s;
}

// VEC elements per access, NV accesses per thread: column (i * threads + t) * VEC
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(1024) k_norm(const NormArgs a) {
  __shared__ float red[2][32];
  const int t = threadIdx.x, threads = blockDim.x, warps = threads >> 5;
  const int H = a.hidden;
  const float root = rsqrtf((float)H);         // squares of v / sqrt(H) are summed: a mean that fits f32 does not overflow
  float post[NV][VEC], pre[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * threads + t) * VEC;
    if (c < H) {
      if (a.post) load_vec<T, VEC>((const T*)a.post + c, post[i]);
      if (a.y) load_vec<T, VEC>((const T*)a.pre + c, pre[i]);
    }
  }
  int buf = 0;
  for (long long r = blockIdx.x; r < a.tokens; r += gridDim.x) {
    float x[NV][VEC], b[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * threads + t) * VEC;
      if (c < H) {
        load_vec<T, VEC>((const T*)a.x + r * a.x_row + c, x[i]);
        if (a.block) load_vec<T, VEC>((const T*)a.block + r * a.block_row + c, b[i]);
      }
    }
    if (a.block) {
      float f = a.res_scale;
      if (a.post) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if ((i * threads + t) * VEC < H) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) ss = fmaf(b[i][j] * root, b[i][j] * root, ss);
          }
        const float rs = rsqrtf(block_add(ss, red[buf], warps) + a.eps);
        buf ^= 1;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j) b[i][j] *= rs * post[i][j];
      }
      if (a.gate && !a.gate_col) f *= Elem<T>::get((const T*)a.gate + r * a.gate_row);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * threads + t) * VEC;
        if (c < H) {
          if (a.gate && a.gate_col) {
            float g[VEC];
            load_vec<T, VEC>((const T*)a.gate + r * a.gate_row + c, g);
#pragma unroll
            for (int j = 0; j < VEC; ++j) b[i][j] *= g[j];
          }
#pragma unroll
          for (int j = 0; j < VEC; ++j) x[i][j] = fmaf(f, b[i][j], x[i][j]);
        }
      }
    }
    if (a.x_out) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * threads + t) * VEC;
        if (c < H) store_vec<T, VEC>((T*)a.x_out + r * a.x_out_row + c, x[i]);
      }
    }
    if (a.y) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if ((i * threads + t) * VEC < H) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) ss = fmaf(x[i][j] * root, x[i][j] * root, ss);
        }
      const float rs = rsqrtf(block_add(ss, red[buf], warps) + a.eps);
      buf ^= 1;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * threads + t) * VEC;
        if (c < H) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) x[i][j] *= rs * pre[i][j];
          store_vec<T, VEC>((T*)a.y + r * a.y_row + c, x[i]);
        }
      }
    }
  }
}

template <typename T, int VEC, int NV>
cudaError_t go(const NormArgs& a, int threads, cudaStream_t s) {
  // as many blocks as the SMs hold at once (2048 threads each), rows in turn
  const long long resident = (long long)device_sm_count() * (2048 / threads > 32 ? 32 : 2048 / threads);
  const int grid = (int)(a.tokens < resident ? a.tokens : resident);
  k_norm<T, VEC, NV><<<grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t pick(const NormArgs& a, bool vec, cudaStream_t s) {
  constexpr int W = 16 / sizeof(T);
  const int chunks = vec ? a.hidden / W : a.hidden;
  // one access per thread up to 512 threads, then more accesses per thread
  int nv = 1;
  while (chunks > nv * (nv < 4 ? 512 : 1024) && nv < 32) nv *= 2;
  const int threads = ((chunks + nv - 1) / nv + 31) / 32 * 32;
  if (vec) {
    switch (nv) {
      case 1: return go<T, W, 1>(a, threads, s);
      case 2: return go<T, W, 2>(a, threads, s);
      case 4: return go<T, W, 4>(a, threads, s);
      default: return go<T, W, 8>(a, threads, s);
    }
  }
  switch (nv) {
    case 1: return go<T, 1, 1>(a, threads, s);
    case 2: return go<T, 1, 2>(a, threads, s);
    case 4: return go<T, 1, 4>(a, threads, s);
    case 8: return go<T, 1, 8>(a, threads, s);
    case 16: return go<T, 1, 16>(a, threads, s);
    default: return go<T, 1, 32>(a, threads, s);
  }
}

}  // namespace

cudaError_t launch_norm(const moe_norm_args& m, cudaStream_t s) {
  if (m.tokens <= 0) return cudaSuccess;
  NormArgs a;
  a.x = m.x_d, a.block = m.block_d, a.post = m.post_w_d, a.gate = m.gate_d, a.pre = m.pre_w_d;
  a.x_out = m.x_out_d, a.y = m.y_d;
  a.tokens = m.tokens, a.hidden = m.hidden;
  a.x_row = m.x_row, a.block_row = m.block_row, a.gate_row = m.gate_row, a.x_out_row = m.x_out_row, a.y_row = m.y_row;
  a.gate_col = m.gate_col, a.res_scale = m.res_scale, a.eps = m.eps;
  const size_t e = m.dtype == MOE_BF16 ? 2 : 4;
  // 16-byte accesses need every row to start on 16 bytes (a gate per row is read alone)
  const bool vec = aligned(16, m.x_d, m.block_d, m.post_w_d, m.pre_w_d, m.x_out_d, m.y_d, m.hidden * e, m.x_row * e,
                           m.block_row * e, m.x_out_row * e, m.y_row * e) &&
                   (!m.gate_d || !m.gate_col || aligned(16, m.gate_d, m.gate_row * e));
  return m.dtype == MOE_BF16 ? pick<__nv_bfloat16>(a, vec, s) : pick<float>(a, vec, s);
}

}  // namespace moe
