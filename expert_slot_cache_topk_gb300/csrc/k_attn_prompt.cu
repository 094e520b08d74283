// Attention over packed prompts in f32 arithmetic, for every type, head size
// (a multiple of 8 up to 256) and alignment.  Causal: query r of a sequence
// with lq queries and lk keys sees the keys j <= r + lk - lq.
//
// k_prompt: a block of 256 threads takes 64 or 32 queries of one head.  Tiles of BN keys
// pass through shared memory (f32: copied as they are, one tile ahead); thread (ty, tx)
// holds the scores of its 4 or 2 rows x BN / 16 keys, the row maxima and sums run over
// the 16 threads of a row, and the weights go through shared memory to the product with
// V, of which the thread holds D / 16 columns of its rows.  What bounds it is shared
// memory, which gives 128 bytes a cycle to registers: a 4 x 4 share reads 32 floats for
// 64 multiply-adds, twice the time of these (26 TFLOP/s for 16 prompts of up to 1000
// tokens, 8 heads of 64, in f32).  k_prompt_keys below: aligned f32, smaller heads.
#include <cmath>

#include "attn_common.cuh"

namespace moe {

cudaError_t launch_attn_prompt_tc(const moe_prompt_args& a, cudaStream_t s);   // k_attn_prompt_tc.cu

namespace {

using namespace attn;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ void cp16(float* to, const float* from, bool real) {
  const int n = real ? 16 : 0;                 // 0: zeros, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from), "r"(n)
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two multiply-adds in one instruction
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ unsigned long long pair(float lo, float hi) {
  unsigned long long v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ float2 unpair(unsigned long long v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ bool not_finite(float v) { return !(fabsf(v) <= 3.4028235e38f); }

// The sequence and the first query of row tile `b` (tiles of `rows` queries).
// Sequence i owns the tiles from starts[i] / rows + i on: enough of them for
// its queries, and no two sequences share one.  Tiles past a sequence's last
// query are empty: *r0 >= its length.
__device__ __forceinline__ int tile_sequence(const int32_t* starts, int n, int b, int rows, int* r0) {
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

template <typename T, int DP, int BM, int BN, bool VEC>
__global__ void __launch_bounds__(256) k_prompt(const moe_prompt_args a) {
  wait_ahead();
  constexpr int PIT = DP + 4;                  // row pitch: 16-byte aligned, rows 4 banks apart
  constexpr int RN = BM / 16, CN = BN / 16, DN = DP / 64;    // rows, keys and 4-column groups of a thread
  constexpr bool kAsync = VEC && sizeof(T) == 4;             // tiles are copied as they are, one ahead
  extern __shared__ float sm[];
  float* Q = sm;                               // [BM][PIT], scaled
  float* P = Q + BM * PIT;                     // [BM][BN + 4]
  float* KV = P + BM * (BN + 4);               // K [BN][PIT], V [BN][PIT]; twice when they are copied ahead
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int h = blockIdx.x % a.heads, kh = h / (a.heads / a.kv_heads), D = a.head_dim;
  int r0;                                      // late tiles, the long ones, first
  const int seq = tile_sequence(a.starts_q_d, a.n, a.q_tokens / BM + a.n - 1 - (int)(blockIdx.x / a.heads), BM, &r0);
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
          odd |= not_finite(v[w]);
          to[r * PIT + d + w] = v[w] * f;
        }
      }
    } else {
      for (int x = tid; x < rows * DP; x += 256) {
        const int r = x / DP, d = x % DP;
        float v = 0.f;
        if (first + r < limit && d < D) v = Elem<T>::get((const T*)base + (first + r) * token + head + d);
        odd |= not_finite(v);
        to[r * PIT + d] = v * f;
      }
    }
    return odd;
  };
  load_tile(Q, a.q_d, a.q_token, h * a.q_head, q0 + r0, q1, BM, a.scale * kLog2e);
  float m[RN], l[RN], o[RN][DN][4];
  const int last_row = r0 + BM < lq ? r0 + BM - 1 : lq - 1;
  const int j_begin = a.window > 0 && r0 + off - a.window + 1 > 0 ? (r0 + off - a.window + 1) / BN * BN : 0;
  const int jend = last_row + off + 1;                      // keys any row of the tile sees: below jend <= lk
  // K and V rows of the tile from key `first` on, as they are in memory
  [[maybe_unused]] auto copy_ahead = [&](int first, int turn) {
    if (first < jend) {
      float* K = KV + turn * 2 * BN * PIT;
      for (int x = tid; x < BN * (DP / 4); x += 256) {
        const int r = x / (DP / 4), d = x % (DP / 4) * 4;
        const bool real = k0 + first + r < k1 && d < D;
        const long long row = real ? (long long)(k0 + first + r) : 0;
        cp16(K + r * PIT + d, (const float*)a.k_d + (real ? row * a.k_token + kh * a.k_head + d : 0), real);
        cp16(K + (BN + r) * PIT + d, (const float*)a.v_d + (real ? row * a.v_token + kh * a.v_head + d : 0), real);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // Copied tiles are not looked at on the way.  A block whose result is not finite
  // goes over its keys once more and carefully: a weight of 0 must not meet a value
  // that is not finite behind the mask.
  for (bool careful = false;; careful = true) {
#pragma unroll
    for (int i = 0; i < RN; ++i) {
      m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < DN; ++j)
#pragma unroll
        for (int w = 0; w < 4; ++w) o[i][j][w] = 0.f;
    }
    if (kAsync) copy_ahead(j_begin, 0);
    for (int j0 = j_begin, turn = 0; j0 < jend; j0 += BN, turn ^= 1) {
      float* K = KV + (kAsync ? turn * 2 * BN * PIT : 0);
      float* V = K + BN * PIT;
      bool any_odd = false;
      if constexpr (kAsync) {
        copy_ahead(j0 + BN, turn ^ 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        if (careful) {
          bool odd = false;
          for (int x = tid; x < BN * DP; x += 256) odd |= not_finite(V[x / DP * PIT + x % DP]);
          any_odd = __syncthreads_or(odd);
        }
      } else {
        __syncthreads();
        load_tile(K, a.k_d, a.k_token, kh * a.k_head, k0 + j0, k1, BN, 1.f);
        any_odd = __syncthreads_or(load_tile(V, a.v_d, a.v_token, kh * a.v_head, k0 + j0, k1, BN, 1.f));
      }
      float s[RN][CN];
#pragma unroll
      for (int i = 0; i < RN; ++i)
#pragma unroll
        for (int c = 0; c < CN; ++c) s[i][c] = 0.f;
#pragma unroll 4
      for (int d = 0; d < DP; d += 4) {
        float4 q[RN], k[CN];
#pragma unroll
        for (int i = 0; i < RN; ++i) q[i] = *reinterpret_cast<const float4*>(Q + (ty * RN + i) * PIT + d);
#pragma unroll
        for (int c = 0; c < CN; ++c) k[c] = *reinterpret_cast<const float4*>(K + (tx + 16 * c) * PIT + d);
#pragma unroll
        for (int i = 0; i < RN; ++i)
#pragma unroll
          for (int c = 0; c < CN; ++c) {
            s[i][c] = fmaf(q[i].x, k[c].x, s[i][c]);
            s[i][c] = fmaf(q[i].y, k[c].y, s[i][c]);
            s[i][c] = fmaf(q[i].z, k[c].z, s[i][c]);
            s[i][c] = fmaf(q[i].w, k[c].w, s[i][c]);
          }
      }
#pragma unroll
      for (int i = 0; i < RN; ++i) {
        const int at = r0 + ty * RN + i + off;                 // the last key this row sees
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
          P[(ty * RN + i) * (BN + 4) + tx + 16 * c] = p;
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
          float4 p[RN];
#pragma unroll
          for (int i = 0; i < RN; ++i) p[i] = *reinterpret_cast<const float4*>(P + (ty * RN + i) * (BN + 4) + c);
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int j = 0; j < DN; ++j) {
              const float4 v = *reinterpret_cast<const float4*>(V + (c + u) * PIT + tx * 4 + 64 * j);
#pragma unroll
              for (int i = 0; i < RN; ++i) {
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
          for (int i = 0; i < RN; ++i) {
            const int at = r0 + ty * RN + i + off, j = j0 + c;
            if (j > at || (a.window > 0 && j <= at - a.window)) continue;
            const float w = P[(ty * RN + i) * (BN + 4) + c];
#pragma unroll
            for (int jj = 0; jj < DN; ++jj)
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                // o's indices stay constants: row i is picked by comparison
                const float add = w * V[c * PIT + tx * 4 + 64 * jj + x];
#pragma unroll
                for (int ii = 0; ii < RN; ++ii)
                  if (ii == i) o[ii][jj][x] += add;
              }
          }
      }
        if (kAsync) __syncthreads();                            // this half is free for the copies after next
    }
    if (!kAsync || careful) break;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    bool lost = false;
#pragma unroll
    for (int i = 0; i < RN; ++i)
#pragma unroll
      for (int j = 0; j < DN; ++j)
#pragma unroll
        for (int w = 0; w < 4; ++w) lost |= not_finite(o[i][j][w]);
    if (!__syncthreads_or(lost)) break;
  }
#pragma unroll
  for (int i = 0; i < RN; ++i) {
    const int r = r0 + ty * RN + i;
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

template <typename T, int DP, int BM, int BN, bool VEC>
cudaError_t go(const moe_prompt_args& a, cudaStream_t s) {
  constexpr int tiles = VEC && sizeof(T) == 4 ? 4 : 2;
  constexpr int smem = ((BM + tiles * BN) * (DP + 4) + BM * (BN + 4)) * 4;
  static bool set[kMaxDevices] = {};
  {
    std::lock_guard<std::mutex> lock(launch_state_mutex());
    const int dev = current_device();
    if (dev < 0) return cudaErrorInvalidDevice;
    if (!set[dev]) {
      const cudaError_t e =
          cudaFuncSetAttribute(k_prompt<T, DP, BM, BN, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      set[dev] = true;
    }
  }
  const long long grid = (long long)a.heads * (a.q_tokens / BM + a.n);
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return launch_following(k_prompt<T, DP, BM, BN, VEC>, (unsigned)grid, 256, smem, s, a);
}

// f32 with heads of up to DP elements, 16-byte aligned.  The four warps of a block share
// 4 RM queries of one head and take their tiles of 32 keys in turn, each with a running
// maximum, sum and output of its own; these are joined at the end.  So a warp waits for
// no other in its loop, a row's chain of tiles is four times shorter than with the whole
// block at one tile, and a lane has a larger share of a tile (RM rows x 4 keys, RM rows x
// DP / 8 columns; two multiply-adds to an instruction, the weights stored twice for that),
// so that shared memory gives each value to more of them.  A warp's K is loaded while it
// works on its V and the other way round.  What bounds it: 30 TFLOP/s with the multiply
// pipe 54% and the issue slots 50% busy; registers leave room for two warps to a scheduler.
template <int DP, int RM>
__global__ void __launch_bounds__(128, DP == 64 ? 2 : 1) k_prompt_keys(const moe_prompt_args a) {
  wait_ahead();
  constexpr int W = 4, PIT = DP + 4, BM = 4 * RM, BK = 32, PP = 2 * BK + 4, NJ = DP / 32;
  constexpr int kWarp = 2 * BK * PIT + BM * PP;              // floats of a warp: K, V, P
  extern __shared__ float sm[];
  float* Q = sm;                                             // [BM][PIT], scaled
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rg = lane >> 3, kg = lane & 7;
  float* K = sm + BM * PIT + warp * kWarp;                   // [BK][PIT]; the warp's output in the end
  float* V = K + BK * PIT;                                   // [BK][PIT]
  float* P = V + BK * PIT;                                   // [BM][PP], each weight twice; maxima and sums in the end
  const int h = blockIdx.x % a.heads, kh = h / (a.heads / a.kv_heads), D = a.head_dim;
  int r0;                                      // late tiles, the long ones, first
  const int seq = tile_sequence(a.starts_q_d, a.n, a.q_tokens / BM + a.n - 1 - (int)(blockIdx.x / a.heads), BM, &r0);
  const int q0 = clampi(a.starts_q_d[seq], 0, a.q_tokens), q1 = clampi(a.starts_q_d[seq + 1], q0, a.q_tokens);
  const int k0 = clampi(a.starts_k_d[seq], 0, a.k_tokens), k1 = clampi(a.starts_k_d[seq + 1], k0, a.k_tokens);
  const int lq = q1 - q0, lk = k1 - k0, off = lk - lq;
  if (r0 < 0 || r0 >= lq) return;
  const int last_row = r0 + BM < lq ? r0 + BM - 1 : lq - 1;
  const int j_begin = a.window > 0 && r0 + off - a.window + 1 > 0 ? (r0 + off - a.window + 1) / BK * BK : 0;
  const int jend = last_row + off + 1;                      // keys any row of the tile sees: below jend <= lk
  auto copy = [&](float* to, const void* base, long long token, long long head, int first) {
    constexpr int kLanes = DP / 4;                           // of a row
    const int r = lane / kLanes, d = lane % kLanes * 4;
    const float* from = (const float*)base + (k0 + first + r) * token + kh * head + d;
    const int rows = d < D ? lk - first - r : 0;
    if (first < jend)
#pragma unroll
      for (int x = 0; x < BK; x += 32 / kLanes)
        cp16(to + (x + r) * PIT + d, x < rows ? from + x * token : (const float*)base, x < rows);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int x = tid; x < BM * (DP / 4); x += W * 32) {
    const int r = x / (DP / 4), d = x % (DP / 4) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < lq && d < D)
      v = *reinterpret_cast<const float4*>((const float*)a.q_d + (q0 + r0 + r) * a.q_token + h * a.q_head + d);
    const float f = a.scale * kLog2e;
    *reinterpret_cast<float4*>(Q + r * PIT + d) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
  }
  // A block whose result is not finite goes over its keys once more and carefully: a
  // weight of 0 must not meet a value that is not finite behind the mask.
  for (bool careful = false;; careful = true) {
    float m[RM], l[RM];
    unsigned long long o[RM][NJ][2];                        // columns in pairs
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) o[i][j][0] = o[i][j][1] = 0ull;
    }
    const int j_first = j_begin + warp * BK;
    copy(K, a.k_d, a.k_token, a.k_head, j_first);
    copy(V, a.v_d, a.v_token, a.v_head, j_first);
    __syncthreads();                                        // Q
    for (int j0 = j_first; j0 < jend; j0 += W * BK) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
      unsigned long long s2[RM][4];                         // sums over the even and the odd elements
#pragma unroll
      for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) s2[i][c] = 0ull;
#pragma unroll 2
      for (int d = 0; d < DP; d += 4) {
        ulonglong2 k[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) k[c] = *reinterpret_cast<const ulonglong2*>(K + (kg + 8 * c) * PIT + d);
#pragma unroll
        for (int i = 0; i < RM; ++i) {
          const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(Q + (rg + 4 * i) * PIT + d);
#pragma unroll
          for (int c = 0; c < 4; ++c) s2[i][c] = fma2(q.y, k[c].y, fma2(q.x, k[c].x, s2[i][c]));
        }
      }
      __syncwarp();
      copy(K, a.k_d, a.k_token, a.k_head, j0 + W * BK);
      const bool crossed = j0 + BK - 1 > r0 + off || (a.window > 0 && j0 <= r0 + BM - 1 + off - a.window);
#pragma unroll
      for (int i = 0; i < RM; ++i) {
        const int at = r0 + rg + 4 * i + off;                // the last key this row sees
        float s[4], mx = m[i];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int j = j0 + kg + 8 * c;
          const float2 v = unpair(s2[i][c]);
          s[c] = v.x + v.y;
          if (crossed && (j > at || (a.window > 0 && j <= at - a.window))) s[c] = -INFINITY;
          mx = fmaxf(mx, s[c]);
        }
#pragma unroll
        for (int x = 1; x < 8; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, x));
        const float base = mx == -INFINITY ? 0.f : mx, f = ex2(m[i] - base);
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float p = ex2(s[c] - base);
          sum += p;
          *reinterpret_cast<float2*>(P + (rg + 4 * i) * PP + 2 * (kg + 8 * c)) = make_float2(p, p);
        }
        l[i] = l[i] * f + sum;                               // of the lane's keys
        m[i] = mx;
#pragma unroll
        for (int j = 0; j < NJ; ++j) o[i][j][0] = mul2(o[i][j][0], pair(f, f)), o[i][j][1] = mul2(o[i][j][1], pair(f, f));
      }
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
      bool odd = false;
      if (careful) {
        for (int x = lane; x < BK * DP; x += 32) odd |= not_finite(V[x / DP * PIT + x % DP]);
        odd = __any_sync(kAll, odd);
      }
      if (!odd) {
#pragma unroll 1
        for (int c = 0; c < BK; c += 4) {
          ulonglong2 v[4][NJ];
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
              v[u][j] = *reinterpret_cast<const ulonglong2*>(V + (c + u) * PIT + kg * 4 + 32 * j);
#pragma unroll
          for (int i = 0; i < RM; ++i) {
#pragma unroll
            for (int u = 0; u < 4; u += 2) {
              const ulonglong2 p = *reinterpret_cast<const ulonglong2*>(P + (rg + 4 * i) * PP + 2 * (c + u));
#pragma unroll
              for (int j = 0; j < NJ; ++j) {
                o[i][j][0] = fma2(p.y, v[u + 1][j].x, fma2(p.x, v[u][j].x, o[i][j][0]));
                o[i][j][1] = fma2(p.y, v[u + 1][j].y, fma2(p.x, v[u][j].y, o[i][j][1]));
              }
            }
          }
        }
      } else {
        // values that are not finite: a weight of 0 must not meet those that the mask hides
#pragma unroll 1
        for (int c = 0; c < BK; ++c)
#pragma unroll
          for (int i = 0; i < RM; ++i) {
            const int at = r0 + rg + 4 * i + off, j = j0 + c;
            if (j > at || (a.window > 0 && j <= at - a.window)) continue;
            const unsigned long long w = *reinterpret_cast<const unsigned long long*>(P + (rg + 4 * i) * PP + 2 * c);
#pragma unroll
            for (int jj = 0; jj < NJ; ++jj) {
              const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(V + c * PIT + kg * 4 + 32 * jj);
              o[i][jj][0] = fma2(w, v.x, o[i][jj][0]);
              o[i][jj][1] = fma2(w, v.y, o[i][jj][1]);
            }
          }
      }
      __syncwarp();
      copy(V, a.v_d, a.v_token, a.v_head, j0 + W * BK);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      const int r = rg + 4 * i;
#pragma unroll
      for (int x = 1; x < 8; x <<= 1) l[i] += __shfl_xor_sync(kAll, l[i], x);
      if (kg == 0) P[r * PP] = m[i], P[r * PP + 1] = l[i];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        ulonglong2 v;
        v.x = o[i][j][0], v.y = o[i][j][1];
        *reinterpret_cast<ulonglong2*>(K + r * PIT + kg * 4 + 32 * j) = v;
      }
    }
    __syncthreads();
    bool lost = false;
    for (int x = tid; x < BM * (DP / 4); x += W * 32) {
      const int r = x / (DP / 4), d = x % (DP / 4) * 4;
      const float* first = sm + BM * PIT;                    // the first warp's K
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, first[w * kWarp + 2 * BK * PIT + r * PP]);
      const float base = M == -INFINITY ? 0.f : M;
      float L = 0.f;
      float4 out = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float* at = first + w * kWarp;
        const float f = ex2(at[2 * BK * PIT + r * PP] - base);
        const float4 v = *reinterpret_cast<const float4*>(at + r * PIT + d);
        L = fmaf(at[2 * BK * PIT + r * PP + 1], f, L);
        out.x = fmaf(v.x, f, out.x), out.y = fmaf(v.y, f, out.y), out.z = fmaf(v.z, f, out.z), out.w = fmaf(v.w, f, out.w);
      }
      const bool some = !(L == 0.f);
      const float f = some ? 1.f / L : 0.f;
      out = some ? make_float4(out.x * f, out.y * f, out.z * f, out.w * f) : make_float4(0.f, 0.f, 0.f, 0.f);
      lost |= not_finite(out.x) || not_finite(out.y) || not_finite(out.z) || not_finite(out.w);
      if (r0 + r >= lq || d >= D) continue;
      float* to = (float*)a.out_d + (long long)(q0 + r0 + r) * a.out_token + h * a.out_head + d;
      to[0] = out.x, to[1] = out.y, to[2] = out.z, to[3] = out.w;
      if (d == 0 && a.lse_d) a.lse_d[(long long)(q0 + r0 + r) * a.heads + h] = some ? base * kLn2 + logf(L) : -INFINITY;
    }
    if (!__syncthreads_or(lost) || careful) break;
  }
}

template <int DP, int RM>
cudaError_t go_keys(const moe_prompt_args& a, cudaStream_t s) {
  constexpr int smem = (4 * RM * (DP + 4) + 4 * (64 * (DP + 4) + 4 * RM * 68)) * 4;
  static bool set[kMaxDevices] = {};
  {
    std::lock_guard<std::mutex> lock(launch_state_mutex());
    const int dev = current_device();
    if (dev < 0) return cudaErrorInvalidDevice;
    if (!set[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(k_prompt_keys<DP, RM>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      set[dev] = true;
    }
  }
  const long long grid = (long long)a.heads * (a.q_tokens / (4 * RM) + a.n);
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return launch_following(k_prompt_keys<DP, RM>, (unsigned)grid, 128, smem, s, a);
}

template <typename T, bool VEC, int BM>
cudaError_t by_dim(const moe_prompt_args& a, cudaStream_t s) {
  constexpr bool ahead = VEC && sizeof(T) == 4;     // twice the tiles: half the keys for the larger heads
  if constexpr (!ahead) {
    if (a.head_dim <= 64) return go<T, 64, BM, 64, VEC>(a, s);
  }
  if constexpr (!ahead || BM == 64) {
    if (a.head_dim <= 128) return go<T, 128, BM, ahead ? 32 : 64, VEC>(a, s);
  }
  return go<T, 256, BM, ahead ? 16 : 32, VEC>(a, s);
}

// 64 rows to a block read shared memory least; while that gives every SM less than
// two blocks, 32 rows spread the work better (a prompt of 2048 tokens, 8 heads of 64:
// 227 us with 64 rows, 202 with 32; 16 of up to 1000: 477 and 597).
//
// Aligned f32: with heads of up to 64, k_prompt_keys takes 477 us to 432 for the 16
// prompts and 203 to 153 for the one.  32 rows to a block use shared memory best; with
// less than two blocks of them for an SM, 16 rows are faster (a prompt of 700 tokens: 36
// us instead of 47; of 2048: 165 instead of 153).  With heads of up to 128 a lane's
// output leaves room for 16 rows only: faster for few blocks (5 prompts of up to 400
// tokens: 71 us instead of 90), slower for many (8 of up to 900: 515 instead of 444).
template <typename T, bool VEC>
cudaError_t by_rows(const moe_prompt_args& a, cudaStream_t s) {
  auto few = [&](int rows) { return (long long)a.heads * (a.q_tokens / rows + a.n) < 2ll * device_sm_count(); };
  if constexpr (VEC && sizeof(T) == 4) {
    if (a.head_dim <= 64) return few(32) ? go_keys<64, 4>(a, s) : go_keys<64, 8>(a, s);
    if (a.head_dim <= 128 && few(64)) return go_keys<128, 4>(a, s);
  }
  return few(64) && !(VEC && sizeof(T) == 4 && a.head_dim <= 128) ? by_dim<T, VEC, 32>(a, s) : by_dim<T, VEC, 64>(a, s);
}

}  // namespace

cudaError_t launch_attn_prompt(const moe_prompt_args& a, cudaStream_t s) {
  if (a.n <= 0 || a.q_tokens <= 0) return cudaSuccess;
  const cudaError_t tc = launch_attn_prompt_tc(a, s);
  if (tc != cudaErrorNotSupported) return tc;
  const long long e = a.dtype == MOE_BF16 ? 2 : 4;
  const bool vec = aligned(16, a.q_d, a.k_d, a.v_d, a.q_token * e, a.q_head * e, a.k_token * e, a.k_head * e,
                           a.v_token * e, a.v_head * e);
  if (a.dtype == MOE_BF16) return vec ? by_rows<__nv_bfloat16, true>(a, s) : by_rows<__nv_bfloat16, false>(a, s);
  return vec ? by_rows<float, true>(a, s) : by_rows<float, false>(a, s);
}

}  // namespace moe
