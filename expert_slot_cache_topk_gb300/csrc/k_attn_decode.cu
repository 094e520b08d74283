// Attention of one new token per sequence over a paged key-value cache:
//   s_t = scale * q . k_t,  o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),
// one pass over the tokens with a running maximum m and sum l: when m grows,
// l and o so far are multiplied by exp(m_old - m_new).
#include <cfloat>
#include <cmath>

#include "attn_common.cuh"

namespace moe {
namespace {

using namespace attn;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

struct Dec {
  const char *k, *v;                 // this layer's pools
  const int32_t *table, *lens, *seqs;
  int32_t* status;
  int num_pages, max_seqs, max_pages, page_shift, kv_heads, D;
  const void* q;
  void* out;
  float* lse;
  long long q_token, q_head, out_token, out_head;
  int n, heads, group, window;
  float scale;
};

// How the work is laid out.  An item is (list entry, key head, chunk of its query
// heads); its tokens are cut into blocks (16, or fewer where a token is large).  All blocks of all items form one
// sequence, entry by entry and head by head, and warp g of the grid takes the `pw`
// blocks from g * pw on, whatever items they belong to: every warp streams the same
// number of bytes for any mix of lengths, without the host knowing them.  A warp
// that has a whole item writes its output; otherwise it leaves its maxima, sums and
// unnormalised outputs in its two slots of the workspace (one for the item that it
// starts in, one for the item that it ends in).  A block of threads joins its warps'
// parts of an item, and where an item spans several blocks the last of them to
// finish joins theirs.  Sums are joined in the order of the tokens, so results do
// not depend on timing.
//
// Each warp keeps its own ring of blocks in shared memory, filled by 16-byte
// asynchronous copies two or more blocks ahead (page numbers one block further
// ahead), so no barrier runs inside the loop.  What bounds it is memory: each key
// and value is read once per chunk of query heads.
constexpr int kMaxWarps = 12;                    // of a block of threads
constexpr int kMaxGrid = 320;                    // blocks of threads, at most (one per SM)
constexpr int kMaxChunk = 16;                    // query heads of an item

struct Work {
  float* slots;                  // [grid * warps][2] slots of chunk * (D + 2) floats, then [grid][2] of the blocks
  unsigned* arrived;             // [kMaxGrid], zero between calls
  int chunk, chunks;             // query heads per item, items per key head
};

// The item at hand and a block of it
struct Cursor {
  int i, hc;                     // list entry; key head * chunks + chunk
  int row, from, len;            // tokens [from, len) of the sequence
  int blk, end;                  // block of tokens, and one past the item's last
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real) {
  const int n = real ? 16 : 0;                     // 0: the 16 bytes become zeros, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// bf16 on the tensor cores: S = Q K^T and O += P V with m16n8k16, the chunk's
// query heads on the 16 rows (rows 8.. unused and their arithmetic left out when
// the chunk has at most 8).  This is not the tcgen05 path: one item has at most 16
// rows, and at 2 bytes a value the products ask for a fraction of the legacy rate.
template <int DP, bool SMALL>
struct Bf16 {
  using T = __nv_bfloat16;
  static constexpr int kWarps = 12;
  static constexpr int kBlock = DP == 128 ? 16 : 32;               // tokens
  static constexpr int kTiles = kBlock / 8;                        // n8 tiles of the scores
  static constexpr int kRow = DP * 2;                              // bytes of a token's key in shared memory
  static constexpr int kStage = 2 * kBlock * kRow;                 // K and V of a block: 8 KB
  static constexpr int kStages = 2;
  uint32_t q[DP / 16][4];
  float o[DP / 8][4], m[2], l[2];

  __device__ __forceinline__ void start(const Dec& a, const Work& w, const Cursor& c, int lane) {
    const int kh = c.hc / w.chunks, g0 = c.hc % w.chunks * w.chunk;
    const int r = lane >> 2, t = lane & 3;
#pragma unroll
    for (int x = 0; x < DP / 16; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int g = r + (y & 1) * 8, d = 16 * x + (y >> 1) * 8 + 2 * t;
        uint32_t v = 0;
        if (g < w.chunk && g0 + g < a.group && d < a.D) {
          const T* p = (const T*)a.q + c.i * a.q_token + (kh * a.group + g0 + g) * a.q_head + d;
          v = (uint32_t) * reinterpret_cast<const unsigned short*>(p) | (uint32_t) * reinterpret_cast<const unsigned short*>(p + 1) << 16;
        }
        q[x][y] = v;
      }
#pragma unroll
    for (int x = 0; x < DP / 8; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) o[x][y] = 0.f;
    m[0] = m[1] = -INFINITY, l[0] = l[1] = 0.f;
  }

  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }

  // one block from shared memory; bit t of `live`: token t counts
  __device__ __forceinline__ void block(uint32_t kt, unsigned live, float scale, int lane) {
    const uint32_t vt = kt + kBlock * kRow;
    float s[kTiles][4];
#pragma unroll
    for (int x = 0; x < kTiles; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) s[x][y] = 0.f;
    const int mat = lane >> 3, mr = lane & 7;                       // ldmatrix: matrix and row of this lane's address
    const uint32_t kbase = kt + ((mat >> 1) * 8 + mr) * kRow;
#pragma unroll
    for (int x = 0; x < DP / 16; ++x) {
      const uint32_t col = ((2 * x + (mat & 1)) ^ mr) << 4;
#pragma unroll
      for (int y = 0; y < kTiles / 2; ++y) {
        uint32_t b[4];
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                     : "r"(kbase + y * 16 * kRow + col));
        mma(s[2 * y], q[x], b[0], b[1]);
        mma(s[2 * y + 1], q[x], b[2], b[3]);
      }
    }
    const int t = lane & 3;
#pragma unroll
    for (int x = 0; x < kTiles; ++x)
#pragma unroll
      for (int y = 0; y < (SMALL ? 2 : 4); ++y) s[x][y] *= scale;
    if (live != (kBlock == 32 ? ~0u : (1u << (kBlock & 31)) - 1u)) {
#pragma unroll
      for (int x = 0; x < kTiles; ++x)
#pragma unroll
        for (int y = 0; y < (SMALL ? 2 : 4); ++y)
          if (!(live >> (8 * x + 2 * t + (y & 1)) & 1u)) s[x][y] = -INFINITY;
    }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int x = 0; x < kTiles; ++x)
#pragma unroll
      for (int y = 0; y < (SMALL ? 2 : 4); ++y) mx[y >> 1] = fmaxf(mx[y >> 1], s[x][y]);
#pragma unroll
    for (int h = 0; h < (SMALL ? 1 : 2); ++h) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(kAll, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(kAll, mx[h], 2));
    }
    // the maximum moves only when weights would pass 2^8: they keep their relative
    // precision, and most blocks leave o alone
    const bool grow = mx[0] > m[0] + 8.f || (m[0] == -INFINITY && mx[0] > -INFINITY) ||
                      (!SMALL && (mx[1] > m[1] + 8.f || (m[1] == -INFINITY && mx[1] > -INFINITY)));
    if (__any_sync(kAll, grow)) {
      float f[2] = {1.f, 1.f};
#pragma unroll
      for (int h = 0; h < (SMALL ? 1 : 2); ++h) {
        const float mn = fmaxf(m[h], mx[h]);
        f[h] = mn == -INFINITY ? 1.f : ex2(m[h] - mn);
        m[h] = mn;
        l[h] *= f[h];
      }
#pragma unroll
      for (int x = 0; x < DP / 8; ++x)
#pragma unroll
        for (int y = 0; y < (SMALL ? 2 : 4); ++y) o[x][y] *= f[y >> 1];
    }
    uint32_t p[kTiles / 2][4];
#pragma unroll
    for (int x = 0; x < kTiles; ++x) p[x / 2][2 * (x & 1) + 1] = 0u;
#pragma unroll
    for (int h = 0; h < (SMALL ? 1 : 2); ++h) {
      const float mb = m[h] == -INFINITY ? 0.f : m[h];
#pragma unroll
      for (int x = 0; x < kTiles; ++x) {
        const float p0 = ex2(s[x][2 * h] - mb), p1 = ex2(s[x][2 * h + 1] - mb);
        l[h] += p0 + p1;
        p[x / 2][2 * (x & 1) + h] = pack_bf16(p0, p1);
      }
    }
    const uint32_t vbase = vt + ((mat & 1) * 8 + mr) * kRow;
#pragma unroll
    for (int x = 0; x < DP / 16; ++x) {
      const uint32_t col = ((2 * x + (mat >> 1)) ^ mr) << 4;
#pragma unroll
      for (int y = 0; y < kTiles / 2; ++y) {
        uint32_t b[4];
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                     : "r"(vbase + y * 16 * kRow + col));
        mma(o[2 * x], p[y], b[0], b[1]);
        mma(o[2 * x + 1], p[y], b[2], b[3]);
      }
    }
  }

  __device__ __forceinline__ void total() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(kAll, l[h], 1);
      l[h] += __shfl_xor_sync(kAll, l[h], 2);
    }
  }
  // f(row of the chunk, first of two columns, value, value), and g(row, m, l)
  template <typename F, typename G>
  __device__ __forceinline__ void each(int rows, int D, int lane, F&& f, G&& g) {
    total();
    const int r = lane >> 2, t = lane & 3;
#pragma unroll
    for (int h = 0; h < (SMALL ? 1 : 2); ++h) {
      if (r + 8 * h >= rows) continue;
#pragma unroll
      for (int x = 0; x < DP / 8; ++x)
        if (8 * x < D) f(r + 8 * h, 8 * x + 2 * t, o[x][2 * h], o[x][2 * h + 1], l[h]);
      if (t == 0) g(r + 8 * h, m[h], l[h]);
    }
  }
};

// f32 (and bf16 of head sizes past 128) on the f32 pipes.  Eight lanes share a
// token: lane e of them holds the 16-byte chunks e, e + 8, ... of its key and value,
// so a warp works on four tokens; every lane group keeps its own running softmax
// and the four are joined when the segment ends.
template <typename T_, int NC, int GC>
struct Plain {
  using T = T_;
  static constexpr int kWarps = 8;
  static constexpr int W = 16 / sizeof(T);
  static constexpr int kRow = NC * 128;
  static constexpr int kBlock = kRow <= 256 ? 16 : 4096 / kRow;
  static constexpr int kStage = 2 * kBlock * kRow;
  static constexpr int kStages = kStage <= 4096 ? 6 : 3;
  float q[GC][NC][W], o[GC][NC][W], m[GC], l[GC];

  __device__ __forceinline__ void start(const Dec& a, const Work& w, const Cursor& c, int lane) {
    const int kh = c.hc / w.chunks, g0 = c.hc % w.chunks * w.chunk, e = lane & 7;
#pragma unroll
    for (int g = 0; g < GC; ++g) {
      m[g] = -INFINITY, l[g] = 0.f;
      const bool on = g < w.chunk && g0 + g < a.group;
      const T* p = (const T*)a.q + c.i * a.q_token + (kh * a.group + (on ? g0 + g : 0)) * a.q_head;
#pragma unroll
      for (int x = 0; x < NC; ++x)
#pragma unroll
        for (int y = 0; y < W; ++y) {
          const int d = (e + 8 * x) * W + y;
          q[g][x][y] = on && d < a.D ? Elem<T>::get(p + d) : 0.f;
          o[g][x][y] = 0.f;
        }
    }
  }
  __device__ __forceinline__ void block(uint32_t kt, unsigned live, float scale, int lane) {
    const int e = lane & 7;
#pragma unroll 1
    for (int t = lane >> 3; t < kBlock; t += 4) {
      float v[NC][W], s[GC];
#pragma unroll
      for (int x = 0; x < NC; ++x) load(kt + t * kRow + (((e + 8 * x) ^ (t & 7)) << 4), v[x]);
#pragma unroll
      for (int g = 0; g < GC; ++g) {
        s[g] = 0.f;
#pragma unroll
        for (int x = 0; x < NC; ++x)
#pragma unroll
          for (int y = 0; y < W; ++y) s[g] = fmaf(q[g][x][y], v[x][y], s[g]);
      }
#pragma unroll
      for (int z = 1; z < 8; z <<= 1)
#pragma unroll
        for (int g = 0; g < GC; ++g) s[g] += __shfl_xor_sync(kAll, s[g], z);
#pragma unroll
      for (int x = 0; x < NC; ++x) load(kt + (kBlock + t) * kRow + (((e + 8 * x) ^ (t & 7)) << 4), v[x]);
      if (live >> t & 1u) {
#pragma unroll
        for (int g = 0; g < GC; ++g) {
          s[g] *= scale;
          if (s[g] > m[g] || m[g] == -INFINITY) {
            const float mn = fmaxf(m[g], s[g]), f = mn == -INFINITY ? 1.f : exp2f(m[g] - mn);
            m[g] = mn, l[g] *= f;
#pragma unroll
            for (int x = 0; x < NC; ++x)
#pragma unroll
              for (int y = 0; y < W; ++y) o[g][x][y] *= f;
          }
          const float p = exp2f(s[g] - (m[g] == -INFINITY ? 0.f : m[g]));
          l[g] += p;
#pragma unroll
          for (int x = 0; x < NC; ++x)
#pragma unroll
            for (int y = 0; y < W; ++y) o[g][x][y] = fmaf(p, v[x][y], o[g][x][y]);
        }
      }
    }
  }
  static __device__ __forceinline__ void load(uint32_t at, float (&v)[W]) {
    uint32_t u[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(at));
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      if constexpr (W == 4) {
        v[y] = __uint_as_float(u[y]);
      } else {
        v[2 * y] = __uint_as_float(u[y] << 16);
        v[2 * y + 1] = __uint_as_float(u[y] & 0xffff0000u);
      }
    }
  }
  template <typename F, typename G>
  __device__ __forceinline__ void each(int rows, int D, int lane, F&& f, G&& put) {
    const int e = lane & 7;
#pragma unroll
    for (int g = 0; g < GC; ++g) {
#pragma unroll
      for (int z = 8; z < 32; z <<= 1) {
        const float mo = __shfl_xor_sync(kAll, m[g], z), lo = __shfl_xor_sync(kAll, l[g], z);
        const float mn = fmaxf(m[g], mo), b = mn == -INFINITY ? 0.f : mn;
        const float mine = exp2f(m[g] - b), other = exp2f(mo - b);
        l[g] = l[g] * mine + lo * other;
#pragma unroll
        for (int x = 0; x < NC; ++x)
#pragma unroll
          for (int y = 0; y < W; ++y) o[g][x][y] = o[g][x][y] * mine + __shfl_xor_sync(kAll, o[g][x][y], z) * other;
        m[g] = mn;
      }
      if (lane < 8 && g < rows) {
#pragma unroll
        for (int x = 0; x < NC; ++x)
          if ((e + 8 * x) * W < D) {
#pragma unroll
            for (int y = 0; y < W; y += 2) f(g, (e + 8 * x) * W + y, o[g][x][y], o[g][x][y + 1], l[g]);
          }
        if (e == 0) put(g, m[g], l[g]);
      }
    }
  }
};

template <typename Op>
__global__ void __launch_bounds__(Op::kWarps * 32, 1) k_decode(const Dec a, const Work w) {
  using T = typename Op::T;
  constexpr int kBlock = Op::kBlock, kWarps = Op::kWarps, kThreads = kWarps * 32;
  extern __shared__ __align__(1024) unsigned char ring[];
  __shared__ long long part[kThreads + 1];           // blocks before each thread's entries
  __shared__ struct { long long first, last; int i, hc; } rec[kWarps][2];
  __shared__ int joins;                              // the item at hand is complete: join it here
  __shared__ long long wsum[kWarps];
  __shared__ unsigned livemask[kWarps][Op::kStages];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int items = a.kv_heads * w.chunks;           // per entry
  const long long cap = (long long)a.max_pages << a.page_shift;

  // the tokens of an entry; nothing for a row out of range
  auto entry = [&](int i, int& row, int& from, int& len) {
    row = a.seqs[i];
    len = (unsigned)row < (unsigned)a.max_seqs ? a.lens[row] : -1;
    if (len < 0 || len > cap) {
      atomicCAS(a.status, MOE_KV_OK, MOE_KV_BAD_SEQ);
      len = 0, row = 0;
    }
    from = a.window > 0 && len > a.window ? len - a.window : 0;
  };
  auto blocks_of = [](int from, int len) { return len > from ? (len + kBlock - 1) / kBlock - from / kBlock : 0; };

  // every block of threads counts all blocks: thread t the entries [t * per, (t + 1) * per)
  const int per = (a.n + kThreads - 1) / kThreads;
  long long mine = 0;
  for (int i = tid * per; i < (tid + 1) * per && i < a.n; ++i) {
    int row, from, len;
    entry(i, row, from, len);
    mine += blocks_of(from, len);
  }
  long long scan = mine;
#pragma unroll
  for (int z = 1; z < 32; z <<= 1) {
    const long long v = __shfl_up_sync(kAll, scan, z);
    if (lane >= z) scan += v;
  }
  if (lane == 31) wsum[warp] = scan;
  __syncthreads();
  long long before = 0, total = 0;
  for (int x = 0; x < kWarps; ++x) {
    if (x < warp) before += wsum[x];
    total += wsum[x];
  }
  part[tid] = before + scan - mine;
  if (tid == 0) part[kThreads] = total;
  rec[warp][0].last = rec[warp][1].last = -1;
  __syncthreads();
  const long long all = total * items;
  const long long warps = (long long)gridDim.x * kWarps;
  long long pw = (all + warps - 1) / warps;          // blocks of a warp
  if (pw < 2) pw = 2;

  // entries without tokens
  for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
    int row, from, len;
    entry(i, row, from, len);
    if (len > from) continue;
    for (int x = tid; x < a.heads * a.D; x += kThreads)
      Elem<T>::put((T*)a.out + i * a.out_token + (x / a.D) * a.out_head + x % a.D, 0.f);
    if (a.lse)
      for (int h = tid; h < a.heads; h += kThreads) a.lse[(size_t)i * a.heads + h] = -INFINITY;
  }

  const long long g = (long long)blockIdx.x * kWarps + warp;
  const long long u0 = g * pw, u1 = u0 + pw < all ? u0 + pw : all;
  const int slot_floats = w.chunk * (a.D + 2);
  float* slots = w.slots + (size_t)g * 2 * slot_floats;

  if (u0 < u1) {
    const uint32_t my_ring = smem_at(ring) + warp * Op::kStages * Op::kStage;
    // the cursor of the next block to load: find the entry that holds block u0
    Cursor c;
    {
      int lo = 0, hi = kThreads;                     // part[lo] * items <= u0 < part[hi] * items
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (part[mid] * items <= u0) lo = mid;
        else hi = mid;
      }
      long long u = u0 - part[lo] * items;
      c.i = lo * per;
      for (; c.i < a.n; ++c.i) {
        entry(c.i, c.row, c.from, c.len);
        const long long nb = (long long)blocks_of(c.from, c.len) * items;
        if (u < nb) break;
        u -= nb;
      }
      const int nb = blocks_of(c.from, c.len);
      c.hc = (int)(u / nb);
      c.end = c.from / kBlock + nb;
      c.blk = c.from / kBlock + (int)(u % nb);
    }
    auto advance = [&](Cursor& x) {
      if (++x.blk < x.end) return;
      if (++x.hc == items) {
        x.hc = 0;
        do {
          ++x.i;
          entry(x.i, x.row, x.from, x.len);
        } while (x.len <= x.from && x.i + 1 < a.n);
        x.end = (x.len + kBlock - 1) / kBlock;
      }
      x.blk = x.from / kBlock;
    };
    // page of token (lane % kBlock) of the cursor's block
    auto page_of = [&](const Cursor& x) {
      const int t = x.blk * kBlock + (lane & (kBlock - 1));
      return t >= x.from && t < x.len ? a.table[(size_t)x.row * a.max_pages + (t >> a.page_shift)] : -2;
    };
    const int units = a.D * (int)sizeof(T) / 16;     // 16-byte chunks of a token's key
    const long long head_bytes = (long long)a.D * sizeof(T) << a.page_shift;
    constexpr int kUnits = Op::kRow / 16;            // of a row in shared memory: the rest becomes zeros
    constexpr int kRows = kUnits < 32 ? 32 / kUnits : 1;                 // rows that the warp copies at once
    int stage = 0;
    auto load = [&](const Cursor& x, int page) {
      const bool good = (unsigned)page < (unsigned)a.num_pages;
      if (page != -2 && !good) atomicCAS(a.status, MOE_KV_OK, MOE_KV_BAD_PAGE);
      const unsigned live = __ballot_sync(kAll, good) & (kBlock == 32 ? ~0u : (1u << (kBlock & 31)) - 1u);
      if (lane == 0) livemask[warp][stage] = live;
      // where the lane's own token is; its address is passed on to the lanes that copy it
      const int t = x.blk * kBlock + (lane & (kBlock - 1));
      const long long own = good ? ((long long)page * a.kv_heads + x.hc / w.chunks) * head_bytes +
                                       (t & ((1 << a.page_shift) - 1)) * (a.D * (int)sizeof(T))
                                 : 0;
      const uint32_t dst = my_ring + stage * Op::kStage;
#pragma unroll
      for (int y = 0; y < kBlock * kUnits / 32; ++y) {
        const int row = kUnits < 32 ? lane / kUnits + y * kRows : y * 32 / kUnits;
        const int u = kUnits < 32 ? lane % kUnits : lane + y * 32 % kUnits;
        const long long off = __shfl_sync(kAll, own, row) + u * 16;
        const bool real = (live >> row & 1u) && u < units;
        const uint32_t to = dst + row * Op::kRow + ((u ^ (row & 7)) << 4);
        cp16(to, real ? a.k + off : a.k, real);
        cp16(to + kBlock * Op::kRow, real ? a.v + off : a.v, real);
      }
      stage = stage + 1 == Op::kStages ? 0 : stage + 1;
    };
    Cursor ld = c;
    long long ul = u0;
    int page = page_of(ld);
    auto load_next = [&]() {
      if (ul < u1) {
        load(ld, page);
        if (++ul < u1) {
          advance(ld);
          page = page_of(ld);
        }
      }
      cp_commit();
    };
#pragma unroll 1
    for (int x = 0; x < Op::kStages - 1; ++x) load_next();

    Op op;
    op.start(a, w, c, lane);
    long long first = u0 - (c.blk - c.from / kBlock);              // the item's first block
    long long seg = u0;                                            // the segment's
    const float scale = a.scale * kLog2e;
    int use = 0;
    for (long long u = u0; u < u1; ++u) {
      load_next();
      cp_wait<Op::kStages - 1>();
      __syncwarp();
      op.block(my_ring + use * Op::kStage, livemask[warp][use], scale, lane);
      __syncwarp();
      use = use + 1 == Op::kStages ? 0 : use + 1;
      const bool item_ends = c.blk + 1 == c.end;
      if (item_ends || u + 1 == u1) {
        const int kh = c.hc / w.chunks, g0 = c.hc % w.chunks * w.chunk;
        const int rows = a.group - g0 < w.chunk ? a.group - g0 : w.chunk;
        if (item_ends && seg == first) {                           // the whole item
          T* to = (T*)a.out + c.i * a.out_token + (long long)(kh * a.group + g0) * a.out_head;
          float* lse = a.lse ? a.lse + (size_t)c.i * a.heads + kh * a.group + g0 : nullptr;
          op.each(rows, a.D, lane,
                  [&](int r, int d, float x, float y, float l) {
                    const float f = l == 0.f ? 0.f : 1.f / l;
                    Elem<T>::put(to + r * a.out_head + d, l == 0.f ? 0.f : x * f);
                    Elem<T>::put(to + r * a.out_head + d + 1, l == 0.f ? 0.f : y * f);
                  },
                  [&](int r, float m, float l) {
                    if (lse) lse[r] = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) * kLn2 + logf(l);
                  });
        } else {
          const int z = seg == u0 ? 0 : 1;
          float* to = slots + z * slot_floats;
          op.each(rows, a.D, lane,
                  [&](int r, int d, float x, float y, float) { *reinterpret_cast<float2*>(to + r * a.D + d) = make_float2(x, y); },
                  [&](int r, float m, float l) { *reinterpret_cast<float2*>(to + w.chunk * a.D + 2 * r) = make_float2(m, l); });
          if (lane == 0) {
            rec[warp][z].first = first, rec[warp][z].last = first + (c.end - c.from / kBlock);
            rec[warp][z].i = c.i, rec[warp][z].hc = c.hc;
          }
        }
        if (u + 1 < u1) {
          advance(c);
          op.start(a, w, c, lane);
          first = seg = u + 1;
        }
      } else {
        ++c.blk;
      }
    }
    cp_wait<0>();
  }
  __threadfence();
  __syncthreads();

  // Items that no single warp had whole: join the block's parts, and the blocks'
  // parts once the last of them is there.  Column pairs over threads; when there
  // are few, groups of threads share the slots (a fixed share each, in order).
  const long long block_first = (long long)blockIdx.x * kWarps * pw;
  float* block_slots = w.slots + (size_t)warps * 2 * slot_floats;
  for (int x = 0; x < 2 * kWarps; ++x) {
    const long long first = rec[x >> 1][x & 1].first, last = rec[x >> 1][x & 1].last;
    if (last < 0) continue;
    const long long x0 = block_first + (x >> 1) * pw;
    if (!(first >= x0 || (x == 0 && first < block_first))) continue;     // an earlier warp has the item's start
    const long long ga = first / pw, gb = (last - 1) / pw;               // the warps that hold parts of it
    const int ca = (int)(ga / kWarps), cb = (int)(gb / kWarps);          // and their blocks
    const int i = rec[x >> 1][x & 1].i, hc = rec[x >> 1][x & 1].hc;
    const int kh = hc / w.chunks, g0 = hc % w.chunks * w.chunk;
    const int rows = a.group - g0 < w.chunk ? a.group - g0 : w.chunk;
    const int pairs = rows * a.D / 2;
    // sums the slots q = from .. to (inclusive) at slot(q); done(column pair, m, l, o, o)
    auto join = [&](long long from, long long to, auto&& slot, auto&& done) {
      int split = 1;
      while (split * 2 * pairs <= kThreads && split * 2 <= to - from + 1) split *= 2;
      float* sh = reinterpret_cast<float*>(ring);                        // [split][pairs][4]: m, l, o, o
      const long long share = (to - from + split) / split;
      for (int y = tid; y < pairs * split; y += kThreads) {
        const int sp = y / pairs, e = y % pairs, r = e / (a.D / 2), d = e % (a.D / 2) * 2;
        const long long q0 = from + sp * share, q1 = q0 + share < to + 1 ? q0 + share : to + 1;
        float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll 8
        for (long long q = q0; q < q1; ++q) m = fmaxf(m, __ldcg(slot(q) + w.chunk * a.D + 2 * r));
        const float b = m == -INFINITY ? 0.f : m;
#pragma unroll 8
        for (long long q = q0; q < q1; ++q) {
          const float* sl = slot(q);
          const float2 ml = __ldcg(reinterpret_cast<const float2*>(sl + w.chunk * a.D + 2 * r));
          const float2 v = __ldcg(reinterpret_cast<const float2*>(sl + r * a.D + d));
          const float f = exp2f(ml.x - b);
          l = fmaf(ml.y, f, l), o0 = fmaf(v.x, f, o0), o1 = fmaf(v.y, f, o1);
        }
        if (split > 1) *reinterpret_cast<float4*>(sh + 4 * y) = make_float4(m, l, o0, o1);
        else done(e, m, l, o0, o1);
      }
      if (split > 1) {
        __syncthreads();
        if (tid < pairs) {
          float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
          for (int q = 0; q < split; ++q) m = fmaxf(m, sh[4 * (tid + q * pairs)]);
          const float b = m == -INFINITY ? 0.f : m;
          for (int q = 0; q < split; ++q) {
            const float4 v = *reinterpret_cast<const float4*>(sh + 4 * (tid + q * pairs));
            const float f = exp2f(v.x - b);
            l = fmaf(v.y, f, l), o0 = fmaf(v.z, f, o0), o1 = fmaf(v.w, f, o1);
          }
          done(tid, m, l, o0, o1);
        }
      }
    };
    auto result = [&](int e, float m, float l, float o0, float o1) {
      const int r = e / (a.D / 2), d = e % (a.D / 2) * 2;
      T* out = (T*)a.out + i * a.out_token + (long long)(kh * a.group + g0 + r) * a.out_head + d;
      const float f = l == 0.f ? 0.f : 1.f / l;
      Elem<T>::put(out, l == 0.f ? 0.f : o0 * f);
      Elem<T>::put(out + 1, l == 0.f ? 0.f : o1 * f);
      if (d == 0 && a.lse)
        a.lse[(size_t)i * a.heads + kh * a.group + g0 + r] = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) * kLn2 + logf(l);
    };
    auto warp_slot = [&](long long q) {                                  // 1: the item starts inside the warp's run
      return w.slots + ((size_t)q * 2 + (first > q * pw ? 1 : 0)) * slot_floats;
    };
    auto block_slot = [&](long long q) {
      return block_slots + ((size_t)q * 2 + (first > q * kWarps * pw ? 1 : 0)) * slot_floats;
    };
    __syncthreads();                                                     // the last item's shared memory is read
    const long long lo = (long long)blockIdx.x * kWarps, hi = lo + kWarps - 1;
    if (ca == cb) {
      join(ga, gb, warp_slot, result);
      continue;
    }
    float* mine = block_slot(blockIdx.x);
    join(ga > lo ? ga : lo, gb < hi ? gb : hi, warp_slot, [&](int e, float m, float l, float o0, float o1) {
      const int r = e / (a.D / 2), d = e % (a.D / 2) * 2;
      *reinterpret_cast<float2*>(mine + r * a.D + d) = make_float2(o0, o1);
      if (d == 0) *reinterpret_cast<float2*>(mine + w.chunk * a.D + 2 * r) = make_float2(m, l);
    });
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      joins = atomicAdd(&w.arrived[ca], 1u) == (unsigned)(cb - ca);
      if (joins) w.arrived[ca] = 0;
      __threadfence();
    }
    __syncthreads();
    if (joins) join(ca, cb, block_slot, result);
  }
}

template <typename Op>
cudaError_t go(const Dec& a, const Work& w, cudaStream_t s) {
  constexpr int smem = Op::kWarps * Op::kStages * Op::kStage;
  static_assert(Op::kWarps <= kMaxWarps, "slots");
  static bool set[kMaxDevices] = {};
  {
    std::lock_guard<std::mutex> lock(launch_state_mutex());
    const int dev = current_device();
    if (dev < 0) return cudaErrorInvalidDevice;
    if (!set[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(k_decode<Op>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      set[dev] = true;
    }
  }
  const int sms = device_sm_count();
  k_decode<Op><<<sms < kMaxGrid ? sms : kMaxGrid, Op::kWarps * 32, smem, s>>>(a, w);
  return cudaGetLastError();
}

// query heads of an item: the group in equal parts of at most `most`
int chunk_of(int group, int most) {
  const int parts = (group + most - 1) / most;
  return (group + parts - 1) / parts;
}

}  // namespace

size_t attn_decode_work_bytes(const moe_kv_pages& kv, int max_heads) {
  const int group = max_heads / kv.kv_heads;
  const int chunk = group < kMaxChunk ? group : kMaxChunk;
  return 2048 + (size_t)kMaxGrid * (kMaxWarps + 1) * 2 * chunk * (kv.head_dim + 2) * 4;
}

cudaError_t launch_attn_decode(const moe_kv_pages& kv, const DecodeArgs& m, cudaStream_t s) {
  if (m.n <= 0) return cudaSuccess;
  Dec a;
  const size_t e = kv.dtype == MOE_BF16 ? 2 : 4;
  const size_t layer = (size_t)kv.num_pages * kv.kv_heads * kv.page_tokens * kv.head_dim * e;
  a.k = (const char*)kv.k_d + m.layer * layer, a.v = (const char*)kv.v_d + m.layer * layer;
  a.table = kv.table_d, a.lens = kv.lens_d, a.seqs = m.seqs, a.status = kv.status_d;
  a.num_pages = kv.num_pages, a.max_seqs = kv.max_seqs, a.max_pages = kv.max_pages;
  a.page_shift = 0;
  while ((1 << a.page_shift) < kv.page_tokens) ++a.page_shift;
  a.kv_heads = kv.kv_heads, a.D = kv.head_dim;
  a.q = m.q, a.out = m.out, a.lse = m.lse;
  a.q_token = m.q_token, a.q_head = m.q_head, a.out_token = m.out_token, a.out_head = m.out_head;
  a.n = m.n, a.heads = m.heads, a.group = m.heads / kv.kv_heads, a.window = m.window, a.scale = m.scale;
  Work w;
  char* work = (char*)kv.work_d + kv_work_bytes(kv);
  static_assert(kMaxGrid * 4 <= 2048, "arrival counts");
  w.arrived = (unsigned*)work;
  w.slots = (float*)(work + 2048);
  const bool tensor = kv.dtype == MOE_BF16 && a.D <= 128;
  w.chunk = chunk_of(a.group, tensor ? kMaxChunk : a.D > 128 ? 2 : 4);
  w.chunks = (a.group + w.chunk - 1) / w.chunk;
  if (tensor) {
    if (a.D <= 64) return w.chunk <= 8 ? go<Bf16<64, true>>(a, w, s) : go<Bf16<64, false>>(a, w, s);
    return w.chunk <= 8 ? go<Bf16<128, true>>(a, w, s) : go<Bf16<128, false>>(a, w, s);
  }
  if (kv.dtype == MOE_BF16) return go<Plain<__nv_bfloat16, 4, 2>>(a, w, s);
  if (a.D <= 32) return go<Plain<float, 1, 4>>(a, w, s);
  if (a.D <= 64) return go<Plain<float, 2, 4>>(a, w, s);
  if (a.D <= 128) return go<Plain<float, 4, 4>>(a, w, s);
  return go<Plain<float, 8, 2>>(a, w, s);
}

}  // namespace moe
