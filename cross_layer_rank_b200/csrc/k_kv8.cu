// KV cache in 8 bits: writing rows into it, single-token attention over it and
// eviction of whole blocks by the attention they had.
//
// A cache holds, per unit (sequence b, KV head h), `capacity` rows of K and of V
// as e4m3 codes; `block` rows share one scale 2^e.  e4m3 is a floating-point
// format, so a power of two costs no precision against a scale of full
// mantissa, and the quotient x / 2^e is exact in f32: the codes follow from the
// rows alone, whatever the order of evaluation.  One scale for all columns of a
// head suits keys, whose channels differ in size, for the same reason: every
// code keeps its own exponent.
#include <cuda_fp8.h>

#include <algorithm>

#include "xkv_common.cuh"
#include "xkv_internal.h"

namespace xkv {
namespace {

constexpr int kDevInvalid = XKV_ERR_INVALID_ARG;  // a length on the device that the cache cannot hold
constexpr int kTile = 128;                        // token rows of one attention tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kScaleExpMin = -117;  // 2^-117 times the least code 2^-9 is the least normal f32

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// Least e >= kScaleExpMin with a <= 448 * 2^e, a = 1.m * 2^x given by its bits
// (finite, >= 0): 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exp(uint32_t a_bits) {
  const int x = static_cast<int>(a_bits >> 23) - 127;
  const int e = x - 8 + ((a_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(e, kScaleExpMin);
}

__device__ __forceinline__ uint16_t to_e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint16_t c) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
}

// A length from the device, held to [0, most]; one outside is recorded.
__device__ __forceinline__ int64_t checked_len(int32_t n, int64_t most, int* status) {
  if (n >= 0 && n <= most) return n;
  record_status(status, kDevInvalid);
  return n < 0 ? 0 : most;
}

// ---------------------------------------------------------------- append
struct AppendArgs {
  const void* src[2];  // K, V rows
  uint8_t* code[2];
  float* scale[2];
  float* weight;
  int32_t* ids;
  const int32_t* lens;
  const int32_t* counts;
  int64_t n_new, row_stride, batch_stride, capacity;
  int Hkv, hd, block, nb;  // nb: blocks that n_new rows can touch
  int* status;
};

// Eight elements of a row as f32.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
  const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf2_to_f2(u[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load8(const float* p, float* x) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// One CTA per (sequence, touched block, K or V, head): the new rows of one block
// are reduced to their largest finite magnitude and rounded; a block that held
// rows keeps the larger of its scale and the new one, its codes re-rounded when
// the scale grows.
template <typename T>
__global__ void __launch_bounds__(256) kv8_append_kernel(const AppendArgs a) {
  __shared__ uint32_t s_max[8];
  const int tid = threadIdx.x, nthr = blockDim.x;
  int64_t i = blockIdx.x;
  const int h = static_cast<int>(i % a.Hkv);
  i /= a.Hkv;
  const int kv = static_cast<int>(i & 1);
  i >>= 1;
  const int j = static_cast<int>(i % a.nb);
  const int b = static_cast<int>(i / a.nb);
  const int64_t len = checked_len(a.lens[b], a.capacity, a.status);
  int64_t count = a.counts ? a.counts[b] : a.n_new;
  if (count < 0 || count > a.n_new || len + count > a.capacity) {
    if (tid == 0) record_status(a.status, kDevInvalid);
    count = max(int64_t(0), min(min(count, a.n_new), a.capacity - len));
  }
  const int64_t blk = len / a.block + j;
  const int64_t lo = blk * a.block;
  const int64_t r0 = max(lo, len), r1 = min(lo + a.block, len + count);
  if (r0 >= r1) return;
  const int64_t unit = static_cast<int64_t>(b) * a.Hkv + h;
  const int vpr = a.hd / 8, nv = static_cast<int>(r1 - r0) * vpr;
  const T* src = static_cast<const T*>(a.src[kv]) + b * a.batch_stride + (r0 - len) * a.row_stride + h * a.hd;
  uint8_t* code = a.code[kv] + (unit * a.capacity + r0) * a.hd;
  uint32_t big = 0;
  for (int v = tid; v < nv; v += nthr) {
    float x[8];
    load8(src + (v / vpr) * a.row_stride + (v % vpr) * 8, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t m = __float_as_uint(x[e]) & 0x7FFFFFFFu;
      big = max(big, m < 0x7F800000u ? m : 0u);
    }
  }
  big = __reduce_max_sync(0xffffffffu, big);
  if ((tid & 31) == 0) s_max[tid >> 5] = big;
  __syncthreads();
  for (int w = 0; w < nthr / 32; ++w) big = max(big, s_max[w]);
  int e = scale_exp(big);
  float* scale = a.scale[kv] + unit * (a.capacity / a.block) + blk;
  const bool started = len > lo;
  if (started) {
    const float was = *scale;
    const float now = fmaxf(was, pow2f(e));
    if (now > was) {
      // the block's scale grows: its codes once more, on the new scale
      const float ratio = was / now;
      uint2* old = reinterpret_cast<uint2*>(a.code[kv] + (unit * a.capacity + lo) * a.hd);
      for (int v = tid; v < static_cast<int>(len - lo) * vpr; v += nthr) {
        const uint2 w = old[v];
        const uint32_t c[2] = {w.x, w.y};
        uint32_t o[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 f0 = from_e4m3x2(static_cast<uint16_t>(c[q])), f1 = from_e4m3x2(static_cast<uint16_t>(c[q] >> 16));
          o[q] = to_e4m3x2(f0.x * ratio, f0.y * ratio) | static_cast<uint32_t>(to_e4m3x2(f1.x * ratio, f1.y * ratio)) << 16;
        }
        old[v] = make_uint2(o[0], o[1]);
      }
    }
    e = static_cast<int>(__float_as_uint(now) >> 23) - 127;
    __syncthreads();  // every thread has read the old scale
  }
  const float inv = pow2f(-e);
  for (int v = tid; v < nv; v += nthr) {
    float x[8];
    load8(src + (v / vpr) * a.row_stride + (v % vpr) * 8, x);
    uint32_t o[2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
      o[q] = to_e4m3x2(x[4 * q] * inv, x[4 * q + 1] * inv) |
             static_cast<uint32_t>(to_e4m3x2(x[4 * q + 2] * inv, x[4 * q + 3] * inv)) << 16;
    reinterpret_cast<uint2*>(code)[v] = make_uint2(o[0], o[1]);
  }
  if (tid == 0) {
    *scale = pow2f(e);
    if (kv == 0 && !started) {
      // a block opened by this call: no attention yet, and the next number
      const int64_t nblk = a.capacity / a.block, held = (len + a.block - 1) / a.block;
      if (a.weight) a.weight[unit * nblk + blk] = 0.f;
      if (a.ids) a.ids[unit * nblk + blk] = (held ? a.ids[unit * nblk + held - 1] + 1 : 0) + static_cast<int32_t>(blk - held);
    }
  }
}

// ------------------------------------------------------------- attention
struct AttendArgs {
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  const void* q;
  const int32_t* lens;
  float* part;   // partial slots: [gq][hd] sums, [gq] maxima, [gq] softmax sums
  float* wpart;  // [unit][tile][sub-block][gq] sums of the tile's weights, or NULL
  float* wref;   // [unit][tile][gq] the maxima they refer to
  float* weight;
  float* out;
  int64_t capacity;
  int B, Hkv, gq, hd, block, tiles_cap;
  int ctas;
  int* status;
};

__host__ __device__ inline int slot_floats(int gq, int hd) { return gq * (hd + 2); }
__host__ __device__ inline int sub_rows(int block) { return block < 32 ? block : 32; }

// Units' tiles stand in one line (sequence, head, tile), and CTA c of n takes a
// contiguous share of it: ragged lengths need no more CTAs than the card runs.
struct Share {
  int lo, hi;
};
__device__ __forceinline__ Share share_of(int total, int n, int c) {
  const int q = total / n, r = total % n;
  Share s;
  s.lo = c * q + min(c, r);
  s.hi = s.lo + q + (c < r ? 1 : 0);
  return s;
}
// The CTA whose share holds tile x.
__device__ __forceinline__ int cta_of(int total, int n, int x) {
  const int q = total / n, r = total % n;
  const int cut = r * (q + 1);
  return x < cut ? x / (q + 1) : r + (x - cut) / q;
}

__device__ __forceinline__ int tiles_of(const AttendArgs& a, int b) {
  return static_cast<int>((checked_len(a.lens[b], a.capacity, a.status) + kTile - 1) / kTile);
}

// By one warp: the number of tiles before sequence b0 (of its heads), and in all.
// With x >= 0: finds the sequence whose tiles hold x instead.
struct Line {
  int before, total, b;
};
__device__ inline Line walk_line(const AttendArgs& a, int b0, int x) {
  const int lane = threadIdx.x & 31;
  Line r{0, 0, a.B};
  bool found = false;
  for (int base = 0; base < a.B; base += 256) {
    int n[8], sum = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int b = base + lane * 8 + k;
      n[k] = b < a.B ? tiles_of(a, b) * a.Hkv : 0;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += n[k];
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    int at = r.total + inc - sum;
    int hit_b = -1, hit_at = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int b = base + lane * 8 + k;
      if (x >= 0 ? (x >= at && x < at + n[k]) : b == b0) {
        hit_b = b;
        hit_at = at;
      }
      at += n[k];
    }
    const unsigned hit = __ballot_sync(0xffffffffu, hit_b >= 0);
    if (hit && !found) {
      const int src = __ffs(hit) - 1;
      r.b = __shfl_sync(0xffffffffu, hit_b, src);
      r.before = __shfl_sync(0xffffffffu, hit_at, src);
      found = true;
    }
    r.total += __shfl_sync(0xffffffffu, inc, 31);
  }
  return r;
}

// A simple form: one thread per token row for the scores, one per column for
// the values.
template <typename T>
__global__ void __launch_bounds__(128) kv8_attend_kernel(const AttendArgs a) {
  extern __shared__ float sm[];
  __shared__ Line s_line;
  __shared__ int s_total;
  __shared__ float s_red[4][16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gq = a.gq, hd = a.hd;
  float* qs = sm;              // [gq][hd]
  float* ps = qs + gq * hd;    // [gq][128]
  if (warp == 0) {
    Line l = walk_line(a, 0, -1);
    const Share s = share_of(l.total, a.ctas, blockIdx.x);
    const int total = l.total;
    if (s.lo < s.hi) l = walk_line(a, 0, s.lo);
    if (lane == 0) {
      s_line = l;
      s_total = total;
    }
  }
  __syncthreads();
  const Share sh = share_of(s_total, a.ctas, blockIdx.x);
  if (sh.lo >= sh.hi) return;
  int b = s_line.b, nt = tiles_of(a, b);
  int h = (sh.lo - s_line.before) / nt, t = (sh.lo - s_line.before) % nt;
  const float c0 = kLog2e / sqrtf(static_cast<float>(hd));
  const int64_t nblk = a.capacity / a.block;
  for (int x = sh.lo; x < sh.hi;) {
    // one unit's run of tiles
    const int64_t unit = static_cast<int64_t>(b) * a.Hkv + h;
    const int64_t len = checked_len(a.lens[b], a.capacity, nullptr);
    const int t1 = min(nt, t + sh.hi - x);
    const int n_run = t1 - t;
    __syncthreads();
    for (int i = tid; i < gq * hd; i += 128)
      qs[i] = to_f(static_cast<const T*>(a.q)[(static_cast<int64_t>(b) * a.Hkv + h) * gq * hd + i]);
    float acc[2][16], m[16], l[16];
#pragma unroll
    for (int g = 0; g < 16; ++g) {
      acc[0][g] = acc[1][g] = l[g] = 0.f;
      m[g] = -INFINITY;
    }
    for (; t < t1; ++t) {
      __syncthreads();
      const int64_t row = static_cast<int64_t>(t) * kTile + tid;
      float s[16];
#pragma unroll
      for (int g = 0; g < 16; ++g) s[g] = 0.f;
      const bool live = row < len;
      if (live) {
        const uint8_t* kr = a.k + (unit * a.capacity + row) * hd;
        for (int j = 0; j < hd; j += 16) {
          const uint4 w = *reinterpret_cast<const uint4*>(kr + j);
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 f = from_e4m3x2(static_cast<uint16_t>(u[e / 2] >> (16 * (e & 1))));
#pragma unroll
            for (int g = 0; g < 16; ++g)
              if (g < gq) s[g] = fmaf(f.x, qs[g * hd + j + 2 * e], fmaf(f.y, qs[g * hd + j + 2 * e + 1], s[g]));
          }
        }
        const float c = c0 * a.k_scale[unit * nblk + row / a.block];
#pragma unroll
        for (int g = 0; g < 16; ++g) s[g] *= c;
      }
#pragma unroll
      for (int g = 0; g < 16; ++g) {
        const float w = warp_max(live ? s[g] : -INFINITY);
        if (lane == 0) s_red[warp][g] = w;
      }
      __syncthreads();
      float* wp = a.wpart ? a.wpart + (unit * a.tiles_cap + t) * (kTile / sub_rows(a.block)) * gq : nullptr;
      const int sub = sub_rows(a.block);
      const float vs = live ? a.v_scale[unit * nblk + row / a.block] : 0.f;
#pragma unroll
      for (int g = 0; g < 16; ++g) {
        if (g >= gq) break;
        const float mt = fmaxf(fmaxf(s_red[0][g], s_red[1][g]), fmaxf(s_red[2][g], s_red[3][g]));
        const float mn = fmaxf(m[g], mt);
        const float al = m[g] == mn ? 1.f : exp2f(m[g] - mn);
        const float p = live ? exp2f(s[g] - mn) : 0.f;
        m[g] = mn;
        acc[0][g] *= al;
        acc[1][g] *= al;
        l[g] = l[g] * al + p;
        ps[g * 128 + tid] = live ? p * vs : 0.f;
        if (wp) {
          float sum = p;
          for (int o = 1; o < sub; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if (tid % sub == 0) wp[(tid / sub) * gq + g] = sum;
          if (tid == 0) a.wref[(unit * a.tiles_cap + t) * gq + g] = mn;
        }
      }
      __syncthreads();
      const int rows = static_cast<int>(min(static_cast<int64_t>(kTile), len - static_cast<int64_t>(t) * kTile));
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const int col = tid + 128 * cc;
        if (col < hd) {
          const uint8_t* vr = a.v + (unit * a.capacity + static_cast<int64_t>(t) * kTile) * hd + col;
          for (int r = 0; r < rows; ++r) {
            const float vv = from_e4m3x2(vr[static_cast<int64_t>(r) * hd]).x;
#pragma unroll
            for (int g = 0; g < 16; ++g)
              if (g < gq) acc[cc][g] = fmaf(ps[g * 128 + r], vv, acc[cc][g]);
          }
        }
      }
    }
    float* slot = a.part + static_cast<int64_t>(unit + blockIdx.x) * slot_floats(gq, hd);
#pragma unroll
    for (int g = 0; g < 16; ++g) {
      if (g >= gq) break;
      const float w = warp_sum(l[g]);
      if (lane == 0) s_red[warp][g] = w;
      for (int cc = 0; cc < 2; ++cc)
        if (tid + 128 * cc < hd) slot[g * hd + tid + 128 * cc] = acc[cc][g];
    }
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int g = 0; g < 16; ++g) {
        if (g >= gq) break;
        slot[gq * hd + g] = m[g];
        slot[gq * hd + gq + g] = s_red[0][g] + s_red[1][g] + s_red[2][g] + s_red[3][g];
      }
    }
    x += n_run;
    if (t == nt) {
      t = 0;
      if (++h == a.Hkv) {
        h = 0;
        do ++b;
        while (b < a.B && (nt = tiles_of(a, b)) == 0);
        if (b >= a.B) break;
      }
    }
  }
}

// Joins a unit's partials: out = sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i.
// CTA (unit, 0) writes the output; CTAs (unit, y > 0) add a share of the blocks'
// weights, sum_g 2^(ref - M_g) wpart / L_g.
__global__ void __launch_bounds__(256) kv8_combine_kernel(const AttendArgs a) {
  __shared__ int s_before, s_total;
  __shared__ float s_m[16], s_l[16];
  const int unit = blockIdx.x, b = unit / a.Hkv, h = unit % a.Hkv, tid = threadIdx.x, gq = a.gq, hd = a.hd;
  if (tid < 32) {
    const Line l = walk_line(a, b, -1);
    if (tid == 0) {
      s_before = l.before;
      s_total = l.total;
    }
  }
  __syncthreads();
  const int nt = tiles_of(a, b);
  float* out = a.out + static_cast<int64_t>(unit) * gq * hd;
  if (nt == 0) {
    if (blockIdx.y == 0)
      for (int i = tid; i < gq * hd; i += 256) out[i] = 0.f;
    return;
  }
  const int x0 = s_before + h * nt;
  const int c0 = cta_of(s_total, a.ctas, x0), c1 = cta_of(s_total, a.ctas, x0 + nt - 1);
  const int sf = slot_floats(gq, hd);
  const float* base = a.part + static_cast<int64_t>(unit) * sf;
  if (tid < gq) {
    float M = -INFINITY;
    for (int c = c0; c <= c1; ++c) M = fmaxf(M, base[static_cast<int64_t>(c) * sf + gq * hd + tid]);
    float L = 0.f;
    for (int c = c0; c <= c1; ++c) {
      const float* s = base + static_cast<int64_t>(c) * sf + gq * hd + tid;
      L += s[gq] * (s[0] == M ? 1.f : exp2f(s[0] - M));
    }
    s_m[tid] = M;
    s_l[tid] = L;
  }
  __syncthreads();
  if (blockIdx.y == 0) {
    for (int i = tid; i < gq * hd; i += 256) {
      const int g = i / hd;
      float o = 0.f;
      for (int c = c0; c <= c1; ++c) {
        const float* s = base + static_cast<int64_t>(c) * sf;
        const float m = s[gq * hd + g];
        o += s[i] * (m == s_m[g] ? 1.f : exp2f(m - s_m[g]));
      }
      out[i] = o / s_l[g];
    }
    return;
  }
  const int64_t nblk = a.capacity / a.block;
  const int n = static_cast<int>((checked_len(a.lens[b], a.capacity, nullptr) + a.block - 1) / a.block);
  const int sub = sub_rows(a.block), spb = a.block / sub, spt = kTile / sub;
  for (int k = (blockIdx.y - 1) * 256 + tid; k < n; k += (gridDim.y - 1) * 256) {
    float w = 0.f;
    const int64_t s0 = static_cast<int64_t>(k) * spb, tile = s0 / spt;
    const float* ref = a.wref + (static_cast<int64_t>(unit) * a.tiles_cap + tile) * gq;
    const float* p = a.wpart + (static_cast<int64_t>(unit) * a.tiles_cap * spt + s0) * gq;
    for (int g = 0; g < gq; ++g) {
      float s = 0.f;
      for (int e = 0; e < spb; ++e) s += p[e * gq + g];
      w += s * exp2f(ref[g] - s_m[g]) / s_l[g];
    }
    a.weight[unit * nblk + k] += w;
  }
}

// ----------------------------------------------------------------- evict
struct EvictArgs {
  uint8_t* code[2];
  float* scale[2];
  float* weight;
  int32_t* ids;
  const int32_t* lens;
  int32_t* lens_out;
  int64_t capacity;
  int Hkv, hd, block, budget, sink, recent;
  int* status;
};
constexpr int kEvictCtas = 8;       // CTAs (one cluster) per unit
constexpr int kEvictThreads = 256;
constexpr int64_t kEvictMaxBlocks = 131072;  // three bit-mask arrays of a unit's blocks in shared memory

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Order of a weight among the evictable blocks as an unsigned number: NaN below
// every number, -0 as 0, and below the protected blocks' 0xFFFFFFFF.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sums of n small counts f(i) into out[], by the whole CTA.
template <typename F>
__device__ inline int block_scan(int n, int* out, int* s_warp, F f) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int carry = 0;
  for (int base = 0; base < n; base += kEvictThreads) {
    const int i = base + tid;
    const int v = i < n ? f(i) : 0;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int add = carry;
    for (int w = 0; w < kEvictThreads / 32; ++w) {
      if (w < warp) add += s_warp[w];
      carry += s_warp[w];
    }
    if (i < n) out[i] = add + inc - v;
    __syncthreads();
  }
  return carry;
}

// Position of the r-th (from 0) set bit of `mask`, by a whole warp.
__device__ __forceinline__ int nth_bit(uint32_t mask, int r) {
  const int lane = threadIdx.x & 31;
  const bool is = ((mask >> lane) & 1u) && __popc(mask & ((1u << lane) - 1u)) == r;
  return __ffs(__ballot_sync(0xffffffffu, is)) - 1;
}

// Last word whose prefix is <= r.
__device__ __forceinline__ int find_word(const int* pref, int lo, int hi, int r) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pref[mid] <= r) lo = mid;
    else hi = mid;
  }
  return lo;
}

// One cluster per unit.  Every CTA selects the `budget` blocks with the largest
// keys itself (radix selection, eight bits a pass, on up to 131072 keys), then
// the warps of the cluster move the kept blocks that stand past the budget into
// the slots set free below it.  Slots read (>= budget - 1) and written (< budget)
// meet only in slot budget - 1, which the last move writes behind a barrier.
__global__ void __launch_bounds__(kEvictThreads) kv8_evict_kernel(const EvictArgs a) {
  extern __shared__ uint32_t s_dyn[];
  __shared__ uint32_t s_hist[256];
  __shared__ int s_warp[kEvictThreads / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % kEvictCtas, unit = blockIdx.x / kEvictCtas, b = unit / a.Hkv;
  const int64_t len = checked_len(a.lens[b], a.capacity, a.status);
  const int n = static_cast<int>((len + a.block - 1) / a.block);
  const bool writes_len = rank == 0 && unit % a.Hkv == 0 && tid == 0;
  if (n <= a.budget) {
    if (writes_len) a.lens_out[b] = static_cast<int32_t>(len);
    return;  // the whole cluster leaves
  }
  const int64_t nblk = a.capacity / a.block;
  const float* weight = a.weight + unit * nblk;
  const int32_t* ids = a.ids + unit * nblk;
  const int last = ids[n - 1];
  auto key = [&](int i) {
    const int id = ids[i];
    const bool safe = id < a.sink || static_cast<int64_t>(id) > static_cast<int64_t>(last) - a.recent || i == n - 1;
    return safe ? 0xFFFFFFFFu : weight_key(weight[i]);
  };
  // the budget-th largest key
  if (tid == 0) {
    s_prefix = 0;
    s_need = a.budget;
  }
  for (int shift = 24; shift >= 0; shift -= 8) {
    s_hist[tid] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix, mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int i = tid; i < n; i += kEvictThreads) {
      const uint32_t u = key(i);
      if ((u & mask) == prefix) atomicAdd(&s_hist[(u >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l holds bins 255 - 8 l .. 248 - 8 l; the first bin, from above, that reaches the need
      uint32_t c[8], sum = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        c[k] = s_hist[255 - 8 * lane - k];
        sum += c[k];
      }
      uint32_t inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      const uint32_t need = static_cast<uint32_t>(s_need);
      uint32_t above = inc - sum;
      if (above < need && inc >= need) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (above < need && above + c[k] >= need) {
            s_prefix = prefix | static_cast<uint32_t>(255 - 8 * lane - k) << shift;
            s_need = static_cast<int>(need - above);
            above = 0xFFFFFFFFu;
          } else if (above != 0xFFFFFFFFu) {
            above += c[k];
          }
        }
      }
    }
    __syncthreads();
  }
  // bit masks: keys above the threshold, and of those equal to it the lowest `need`
  const uint32_t threshold = s_prefix;
  const int need = s_need;
  const int nw = (n + 31) / 32;
  uint32_t* keep = s_dyn;
  int* pref_a = reinterpret_cast<int*>(s_dyn + nw);
  uint32_t* equal = s_dyn + 2 * nw;
  for (int w = warp; w < nw; w += kEvictThreads / 32) {
    const int i = w * 32 + lane;
    const uint32_t u = i < n ? key(i) : 0u;
    const unsigned gt = __ballot_sync(0xffffffffu, i < n && u > threshold);
    const unsigned eq = __ballot_sync(0xffffffffu, i < n && u == threshold);
    if (lane == 0) {
      keep[w] = gt;
      equal[w] = eq;
    }
  }
  __syncthreads();
  cluster_sync();  // every CTA of the unit has read its keys: the arrays may change from here
  block_scan(nw, pref_a, s_warp, [&](int w) { return __popc(equal[w]); });
  for (int w = tid; w < nw; w += kEvictThreads) {
    int take = need - pref_a[w];
    uint32_t eq = equal[w], add = 0;
    while (take > 0 && eq) {
      add |= eq & (0u - eq);
      eq &= eq - 1;
      --take;
    }
    keep[w] |= add;
  }
  __syncthreads();
  // movers: kept, slot >= budget - 1; free: not kept, slot < budget - 1, and slot budget - 1
  const int edge = a.budget - 1, we = edge / 32;
  const uint32_t below = (1u << (edge & 31)) - 1u;
  auto mover = [&](int w) { return w < we ? 0u : w == we ? keep[w] & ~below : keep[w]; };
  auto empty = [&](int w) { return w < we ? ~keep[w] : (~keep[w] & below) | (1u << (edge & 31)); };
  int* pref_m = pref_a;
  int* pref_f = reinterpret_cast<int*>(equal);
  const int moves = block_scan(nw, pref_m, s_warp, [&](int w) { return __popc(mover(w)); });
  block_scan(we + 1, pref_f, s_warp, [&](int w) { return __popc(empty(w)); });
  const int nv = a.block * a.hd / 16;
  auto move = [&](int r, int first, int step) {
    const int wm = find_word(pref_m, 0, nw, r), wf = find_word(pref_f, 0, we + 1, r);
    const int64_t src = wm * 32 + nth_bit(mover(wm), r - pref_m[wm]);
    const int64_t dst = wf * 32 + nth_bit(empty(wf), r - pref_f[wf]);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint4* from = reinterpret_cast<const uint4*>(a.code[x] + (unit * a.capacity + src * a.block) * a.hd);
      uint4* to = reinterpret_cast<uint4*>(a.code[x] + (unit * a.capacity + dst * a.block) * a.hd);
#pragma unroll 8
      for (int v = first; v < nv; v += step) to[v] = from[v];
    }
    if (first == 0) {
      const int64_t o = unit * nblk;
      a.scale[0][o + dst] = a.scale[0][o + src];
      a.scale[1][o + dst] = a.scale[1][o + src];
      a.weight[o + dst] = a.weight[o + src];
      a.ids[o + dst] = a.ids[o + src];
    }
  };
  for (int r = warp * kEvictCtas + rank; r < moves - 1; r += kEvictCtas * kEvictThreads / 32) move(r, lane, 32);
  cluster_sync();  // slot budget - 1 has been read
  if (rank == 0) move(moves - 1, tid, kEvictThreads);
  if (writes_len) a.lens_out[b] = static_cast<int32_t>(len - static_cast<int64_t>(n - a.budget) * a.block);
}

}  // namespace

// -------------------------------------------------------------- launchers
xkv_status kv8_append_launch(const xkv_kv8_params* p, const xkv_kv8_cache* c, const int32_t* lens,
                             const int32_t* counts, int64_t n_new, xkv_dtype dt, const void* k_new, const void* v_new,
                             int64_t row_stride, int64_t batch_stride, cudaStream_t st) {
  AppendArgs a{};
  a.src[0] = k_new;
  a.src[1] = v_new;
  a.code[0] = static_cast<uint8_t*>(c->k);
  a.code[1] = static_cast<uint8_t*>(c->v);
  a.scale[0] = c->k_scale;
  a.scale[1] = c->v_scale;
  a.weight = c->weight;
  a.ids = c->ids;
  a.lens = lens;
  a.counts = counts;
  a.n_new = n_new;
  a.row_stride = row_stride;
  a.batch_stride = batch_stride;
  a.capacity = p->capacity;
  a.Hkv = p->n_kv_heads;
  a.hd = p->head_dim;
  a.block = p->block;
  const int64_t nb = (n_new + p->block - 2) / p->block + 1;
  a.nb = static_cast<int>(std::min(nb, p->capacity / p->block));
  a.status = device_status_ptr();
  const int64_t grid = static_cast<int64_t>(p->batch) * p->n_kv_heads * 2 * a.nb;
  if (grid > 0x7FFFFFFF) return XKV_ERR_UNSUPPORTED;
  const int64_t vecs = std::min<int64_t>(n_new, p->block) * p->head_dim / 8;
  const int threads = vecs <= 128 ? 128 : 256;
  if (dt == XKV_BF16)
    kv8_append_kernel<__nv_bfloat16><<<static_cast<unsigned>(grid), threads, 0, st>>>(a);
  else
    kv8_append_kernel<float><<<static_cast<unsigned>(grid), threads, 0, st>>>(a);
  return cudaPeekAtLastError() == cudaSuccess ? XKV_OK : XKV_ERR_CUDA;
}

KV8Plan kv8_plan(const xkv_kv8_params* p, int n_q_heads) {
  KV8Plan r{};
  const int gq = n_q_heads / p->n_kv_heads, hd = p->head_dim;
  const int64_t units = static_cast<int64_t>(p->batch) * p->n_kv_heads;
  r.tiles_cap = (p->capacity + kTile - 1) / kTile;
  r.ctas = 8 * num_sms();
  const int spt = kTile / sub_rows(p->block);
  const size_t slots = static_cast<size_t>(units + r.ctas);
  r.off_wpart = align_up(slots * slot_floats(gq, hd) * 4);
  r.off_wref = r.off_wpart + align_up(static_cast<size_t>(units) * r.tiles_cap * spt * gq * 4);
  r.bytes = r.off_wref + align_up(static_cast<size_t>(units) * r.tiles_cap * gq * 4);
  return r;
}

xkv_status kv8_attend_launch(const xkv_kv8_params* p, const xkv_kv8_cache* c, const int32_t* lens, int n_q_heads,
                             xkv_dtype dt, const void* q, float* out, int accumulate, const KV8Plan& plan, void* ws,
                             cudaStream_t st) {
  AttendArgs a{};
  a.k = static_cast<const uint8_t*>(c->k);
  a.v = static_cast<const uint8_t*>(c->v);
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.q = q;
  a.lens = lens;
  char* w = static_cast<char*>(ws);
  a.part = reinterpret_cast<float*>(w);
  if (accumulate) {
    a.wpart = reinterpret_cast<float*>(w + plan.off_wpart);
    a.wref = reinterpret_cast<float*>(w + plan.off_wref);
    a.weight = c->weight;
  }
  a.out = out;
  a.capacity = p->capacity;
  a.B = p->batch;
  a.Hkv = p->n_kv_heads;
  a.gq = n_q_heads / p->n_kv_heads;
  a.hd = p->head_dim;
  a.block = p->block;
  a.tiles_cap = static_cast<int>(plan.tiles_cap);
  a.ctas = plan.ctas;
  a.status = device_status_ptr();
  const size_t smem = static_cast<size_t>(a.gq) * (a.hd + kTile) * 4;
  if (dt == XKV_BF16)
    kv8_attend_kernel<__nv_bfloat16><<<plan.ctas, 128, smem, st>>>(a);
  else
    kv8_attend_kernel<float><<<plan.ctas, 128, smem, st>>>(a);
  int wy = 0;
  if (accumulate) {
    const int64_t nblk = p->capacity / p->block;
    wy = static_cast<int>(std::min<int64_t>((nblk + 255) / 256, 64));
  }
  kv8_combine_kernel<<<dim3(static_cast<unsigned>(p->batch) * p->n_kv_heads, 1 + wy), 256, 0, st>>>(a);
  return cudaPeekAtLastError() == cudaSuccess ? XKV_OK : XKV_ERR_CUDA;
}

xkv_status kv8_evict_launch(const xkv_kv8_params* p, const xkv_kv8_cache* c, const int32_t* lens, int budget, int sink,
                            int recent, int32_t* lens_out, cudaStream_t st) {
  const int64_t nblk = p->capacity / p->block;
  if (nblk > kEvictMaxBlocks) return XKV_ERR_UNSUPPORTED;
  EvictArgs a{};
  a.code[0] = static_cast<uint8_t*>(c->k);
  a.code[1] = static_cast<uint8_t*>(c->v);
  a.scale[0] = c->k_scale;
  a.scale[1] = c->v_scale;
  a.weight = c->weight;
  a.ids = c->ids;
  a.lens = lens;
  a.lens_out = lens_out;
  a.capacity = p->capacity;
  a.Hkv = p->n_kv_heads;
  a.hd = p->head_dim;
  a.block = p->block;
  a.budget = budget;
  a.sink = sink;
  a.recent = recent;
  a.status = device_status_ptr();
  const size_t smem = static_cast<size_t>((nblk + 31) / 32) * 3 * 4;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p->batch) * p->n_kv_heads * kEvictCtas);
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kEvictCtas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kv8_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kEvictMaxBlocks / 32 * 3 * 4)) != cudaSuccess)
    return XKV_ERR_CUDA;
  if (cudaLaunchKernelEx(&cfg, kv8_evict_kernel, a) != cudaSuccess) return XKV_ERR_CUDA;
  return cudaPeekAtLastError() == cudaSuccess ? XKV_OK : XKV_ERR_CUDA;
}

}  // namespace xkv
