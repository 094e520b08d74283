// Attention over packed prompts in f32 arithmetic, for every type, head size
// (a multiple of 8 up to 256) and alignment.  Causal: query r of a sequence
// with lq queries and lk keys sees the keys j <= r + lk - lq.
//
// A block of 256 threads takes 64 queries of one head.  Tiles of BN keys pass
// through shared memory; thread (ty, tx) holds the scores of 4 rows x BN / 16
// keys, the row maxima and sums run over the 16 threads of a row, and the
// weights go through shared memory to the product with V, of which the thread
// holds 4 rows x D / 16 columns.  Two multiply-adds per loaded word and FFMA
// alone: what bounds it is the f32 pipe and shared-memory bandwidth.
#include <cmath>

#include "attn_common.cuh"

namespace moe {

cudaError_t launch_attn_prompt_tc(const moe_prompt_args& a, cudaStream_t s);   // k_attn_prompt_tc.cu

namespace {

using namespace attn;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kBM = 64;

// The sequence and the first query of row tile `b` (tiles of `rows` queries).
// Sequence i owns the tiles from starts[i] / rows + i on: enough of them for
// its queries, and no two sequences share one.  Tiles past a sequence's last
// query are empty: *r0 >= its length.
__device__ __forceinline__ int tile_sequence(const int32_t* __restrict__ starts, int n, int b, int rows, int* r0) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] / rows + mid <= b) lo = mid;
    else hi = mid;
  }
  *r0 = (b - starts[lo] / rows - lo) * rows;
  return lo;
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

template <typename T, int DP, int BN, bool VEC>
__global__ void __launch_bounds__(256) k_prompt(const moe_prompt_args a) {
  constexpr int PIT = DP + 4;                  // row pitch: 16-byte aligned, rows 4 banks apart
  constexpr int CN = BN / 16, DN = DP / 64;    // keys and 4-column groups of a thread
  extern __shared__ float sm[];
  float* Q = sm;                               // [64][PIT], scaled
  float* K = Q + kBM * PIT;                    // [BN][PIT]
  float* V = K + BN * PIT;                     // [BN][PIT]
  float* P = V + BN * PIT;                     // [64][BN + 4]
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int h = blockIdx.x % a.heads, kh = h / (a.heads / a.kv_heads), D = a.head_dim;
  int r0;
  const int seq = tile_sequence(a.starts_q_d, a.n, (int)(blockIdx.x / a.heads), kBM, &r0);
  const int q0 = clampi(a.starts_q_d[seq], 0, a.q_tokens), q1 = clampi(a.starts_q_d[seq + 1], q0, a.q_tokens);
  const int k0 = clampi(a.starts_k_d[seq], 0, a.k_tokens), k1 = clampi(a.starts_k_d[seq + 1], k0, a.k_tokens);
  const int lq = q1 - q0, lk = k1 - k0, off = lk - lq;
  if (r0 < 0 || r0 >= lq) return;
  auto load_tile = [&](float* to, const void* base, long long token, long long head, int first, int limit, int rows,
                       float f) {
    // rows first .. first + rows - 1 (zeros past `limit`); true if this thread met a value that is not finite
    bool odd = false;
    if (VEC) {
      constexpr int W = 16 / sizeof(T);
      for (int x = tid; x < rows * (DP / W); x += 256) {
        const int r = x / (DP / W), d = x % (DP / W) * W;
        float v[W];
#pragma unroll
        for (int w = 0; w < W; ++w) v[w] = 0.f;
        if (first + r < limit && d < D) load_vec<T, W>((const T*)base + (first + r) * token + head + d, v);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          odd |= !(fabsf(v[w]) <= 3.4028235e38f);
          to[r * PIT + d + w] = v[w] * f;
        }
      }
    } else {
      for (int x = tid; x < rows * DP; x += 256) {
        const int r = x / DP, d = x % DP;
        float v = 0.f;
        if (first + r < limit && d < D) v = Elem<T>::get((const T*)base + (first + r) * token + head + d);
        odd |= !(fabsf(v) <= 3.4028235e38f);
        to[r * PIT + d] = v * f;
      }
    }
    return odd;
  };
  load_tile(Q, a.q_d, a.q_token, h * a.q_head, q0 + r0, q1, kBM, a.scale * kLog2e);
  float m[4], l[4], o[4][DN][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < DN; ++j)
#pragma unroll
      for (int w = 0; w < 4; ++w) o[i][j][w] = 0.f;
  }
  const int last_row = r0 + kBM < lq ? r0 + kBM - 1 : lq - 1;
  int j0 = a.window > 0 && r0 + off - a.window + 1 > 0 ? (r0 + off - a.window + 1) / BN * BN : 0;
  const int jend = last_row + off + 1;                      // keys any row of the tile sees: below jend <= lk
  for (; j0 < jend; j0 += BN) {
    __syncthreads();
    load_tile(K, a.k_d, a.k_token, kh * a.k_head, k0 + j0, k1, BN, 1.f);
    const bool odd = load_tile(V, a.v_d, a.v_token, kh * a.v_head, k0 + j0, k1, BN, 1.f);
    const bool any_odd = __syncthreads_or(odd);
    float s[4][CN];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < CN; ++c) s[i][c] = 0.f;
#pragma unroll 4
    for (int d = 0; d < DP; d += 4) {
      float4 q[4], k[CN];
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const float4*>(Q + (ty * 4 + i) * PIT + d);
#pragma unroll
      for (int c = 0; c < CN; ++c) k[c] = *reinterpret_cast<const float4*>(K + (tx + 16 * c) * PIT + d);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < CN; ++c) {
          s[i][c] = fmaf(q[i].x, k[c].x, s[i][c]);
          s[i][c] = fmaf(q[i].y, k[c].y, s[i][c]);
          s[i][c] = fmaf(q[i].z, k[c].z, s[i][c]);
          s[i][c] = fmaf(q[i].w, k[c].w, s[i][c]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = r0 + ty * 4 + i + off;                 // the last key this row sees
      float mx = m[i];
#pragma unroll
      for (int c = 0; c < CN; ++c) {
        const int j = j0 + tx + 16 * c;
        if (j > at || (a.window > 0 && j <= at - a.window)) s[i][c] = -INFINITY;
        mx = fmaxf(mx, s[i][c]);
      }
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, x));
      const float base = mx == -INFINITY ? 0.f : mx, f = exp2f(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < CN; ++c) {
        const float p = exp2f(s[i][c] - base);
        sum += p;
        P[(ty * 4 + i) * (BN + 4) + tx + 16 * c] = p;
      }
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) sum += __shfl_xor_sync(kAll, sum, x);
      l[i] = l[i] * f + sum;
      m[i] = mx;
#pragma unroll
      for (int j = 0; j < DN; ++j)
#pragma unroll
        for (int w = 0; w < 4; ++w) o[i][j][w] *= f;
    }
    __syncwarp();                                           // a row's weights stay within its half warp
    if (!any_odd) {
      for (int c = 0; c < BN; c += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(P + (ty * 4 + i) * (BN + 4) + c);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int j = 0; j < DN; ++j) {
            const float4 v = *reinterpret_cast<const float4*>(V + (c + u) * PIT + tx * 4 + 64 * j);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float w = u == 0 ? p[i].x : u == 1 ? p[i].y : u == 2 ? p[i].z : p[i].w;
              o[i][j][0] = fmaf(w, v.x, o[i][j][0]);
              o[i][j][1] = fmaf(w, v.y, o[i][j][1]);
              o[i][j][2] = fmaf(w, v.z, o[i][j][2]);
              o[i][j][3] = fmaf(w, v.w, o[i][j][3]);
            }
          }
      }
    } else {
      // values that are not finite: a weight of 0 must not meet those that the mask hides
      for (int c = 0; c < BN; ++c)
        for (int i = 0; i < 4; ++i) {
          const int at = r0 + ty * 4 + i + off, j = j0 + c;
          if (j > at || (a.window > 0 && j <= at - a.window)) continue;
          const float w = P[(ty * 4 + i) * (BN + 4) + c];
#pragma unroll
          for (int jj = 0; jj < DN; ++jj)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              // o's indices stay constants: row i is picked by comparison
              const float add = w * V[c * PIT + tx * 4 + 64 * jj + x];
#pragma unroll
              for (int ii = 0; ii < 4; ++ii)
                if (ii == i) o[ii][jj][x] += add;
            }
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + ty * 4 + i;
    if (r >= lq) continue;
    const bool some = !(l[i] == 0.f);
    const float f = some ? 1.f / l[i] : 0.f;
    T* to = (T*)a.out_d + (long long)(q0 + r) * a.out_token + h * a.out_head;
#pragma unroll
    for (int j = 0; j < DN; ++j)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int d = tx * 4 + 64 * j + w;
        if (d < D) Elem<T>::put(to + d, some ? o[i][j][w] * f : 0.f);
      }
    if (tx == 0 && a.lse_d)
      a.lse_d[(long long)(q0 + r) * a.heads + h] = some ? (m[i] == -INFINITY ? 0.f : m[i]) * kLn2 + logf(l[i]) : -INFINITY;
  }
}

template <typename T, int DP, int BN, bool VEC>
cudaError_t go(const moe_prompt_args& a, cudaStream_t s) {
  constexpr int smem = ((kBM + 2 * BN) * (DP + 4) + kBM * (BN + 4)) * 4;
  static bool set[kMaxDevices] = {};
  {
    std::lock_guard<std::mutex> lock(launch_state_mutex());
    const int dev = current_device();
    if (dev < 0) return cudaErrorInvalidDevice;
    if (!set[dev]) {
      const cudaError_t e =
          cudaFuncSetAttribute(k_prompt<T, DP, BN, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      set[dev] = true;
    }
  }
  const long long grid = (long long)a.heads * (a.q_tokens / kBM + a.n);
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  k_prompt<T, DP, BN, VEC><<<(unsigned)grid, 256, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, bool VEC>
cudaError_t by_dim(const moe_prompt_args& a, cudaStream_t s) {
  if (a.head_dim <= 64) return go<T, 64, 64, VEC>(a, s);
  if (a.head_dim <= 128) return go<T, 128, 64, VEC>(a, s);
  return go<T, 256, 32, VEC>(a, s);
}

}  // namespace

cudaError_t launch_attn_prompt(const moe_prompt_args& a, cudaStream_t s) {
  if (a.n <= 0 || a.q_tokens <= 0) return cudaSuccess;
  const cudaError_t tc = launch_attn_prompt_tc(a, s);
  if (tc != cudaErrorNotSupported) return tc;
  const long long e = a.dtype == MOE_BF16 ? 2 : 4;
  const bool vec = aligned(16, a.q_d, a.k_d, a.v_d, a.q_token * e, a.q_head * e, a.k_token * e, a.k_head * e,
                           a.v_token * e, a.v_head * e);
  if (a.dtype == MOE_BF16) return vec ? by_dim<__nv_bfloat16, true>(a, s) : by_dim<__nv_bfloat16, false>(a, s);
  return vec ? by_dim<float, true>(a, s) : by_dim<float, false>(a, s);
}

}  // namespace moe
