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
#include <cmath>
#include <type_traits>

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

// Programmatic launches: let the next kernel begin, and wait for the earlier ones.
// Every block waits, so that a kernel's end stands for the end of all before it.
// What an earlier kernel may write is read with plain loads, not read-only ones:
// it can still be running when this kernel starts.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_earlier() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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
  int B, Hkv, hd, block_log2, nb;  // nb: blocks that n_new rows can touch
  uint32_t vpr_magic;           // ceil(2^20 / (hd / 16)): exact for the quotients of up to 2048 vectors by up to 16
  int* status;
};

// Sixteen elements of a row as they were loaded, and as f32.
template <typename T>
struct Raw16;
template <>
struct Raw16<__nv_bfloat16> {
  uint4 w[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    w[0] = reinterpret_cast<const uint4*>(p)[0];
    w[1] = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ float4 quad(int q) const {  // elements 4 q .. 4 q + 3
    const uint4& u = w[q >> 1];
    const float2 a = bf2_to_f2(q & 1 ? u.z : u.x), b = bf2_to_f2(q & 1 ? u.w : u.y);
    return make_float4(a.x, a.y, b.x, b.y);
  }
};
template <>
struct Raw16<float> {
  float4 w[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = reinterpret_cast<const float4*>(p)[i];
  }
  __device__ __forceinline__ float4 quad(int q) const { return w[q]; }
};

// W warps (1, 4 or 8) per (sequence, touched block, K or V, head): the new rows of
// one block are read once, NV groups of sixteen elements a thread, reduced to
// their largest finite magnitude and rounded; a block that held rows keeps the
// larger of its scale and the new one, its codes re-rounded when the scale grows.
// Small blocks go to a warp each, four to a CTA: 16.6 thousand blocks of 8 x 48
// take 8.7 us, and took 20 with a CTA each.
// Bound by HBM for prompts: four of 64K tokens, 8 heads of 128 (1.61 GB), take
// 238 to 265 us as the card warms up, 6.8 to 6.1 TB/s, a plain copy's rate; one
// token for 32 sequences takes 2.1 us, a launch.  A part-filled block whose scale
// grows costs its own codes a read and a write by the same warps, a vector a lane
// at a time: one token for 32 sequences, 8 heads of 128, blocks of 64, every
// block growing, takes 1.1 us more with blocks half full and 2.8 with full ones;
// blocks of 128 x 256, 4.1 and 8.6.
constexpr int append_threads(int W) { return W == 8 ? 256 : 128; }

template <typename T, int NV, int W>
__global__ void __launch_bounds__(append_threads(W)) kv8_append_kernel(const AppendArgs a) {
  __shared__ uint32_t s_max[8];
  constexpr int nthr = 32 * W;
  const int tid = threadIdx.x & (nthr - 1);
  let_next_start();
  int64_t i = static_cast<int64_t>(blockIdx.x) * (append_threads(W) / nthr) + threadIdx.x / nthr;
  const int h = static_cast<int>(i % a.Hkv);
  i /= a.Hkv;
  const int kv = static_cast<int>(i & 1);
  i >>= 1;
  const int j = static_cast<int>(i % a.nb);
  const int b = static_cast<int>(i / a.nb);
  wait_for_earlier();
  if (b >= a.B) return;
  const int64_t len = checked_len(a.lens[b], a.capacity, a.status);
  int64_t count = a.counts ? a.counts[b] : a.n_new;
  if (count < 0 || count > a.n_new || len + count > a.capacity) {
    if (tid == 0) record_status(a.status, kDevInvalid);
    count = max(int64_t(0), min(min(count, a.n_new), a.capacity - len));
  }
  const int64_t blk = (len >> a.block_log2) + j;
  const int64_t lo = blk << a.block_log2;
  const int64_t r0 = max(lo, len), r1 = min(lo + (1 << a.block_log2), len + count);
  if (r0 >= r1) return;
  const int64_t unit = static_cast<int64_t>(b) * a.Hkv + h, nblk = a.capacity >> a.block_log2;
  const int vpr = a.hd / 16, nv = static_cast<int>(r1 - r0) * vpr;
  const T* src = static_cast<const T*>(a.src[kv]) + b * a.batch_stride + (r0 - len) * a.row_stride + h * a.hd;
  Raw16<T> raw[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int v = tid + k * nthr;
    if (v < nv) {
      const int row = static_cast<int>((static_cast<uint32_t>(v) * a.vpr_magic) >> 20);  // v / vpr
      raw[k].load(src + row * a.row_stride + (v - row * vpr) * 16);
    }
  }
  float* scale = a.scale[kv] + unit * nblk + blk;
  const bool started = len > lo;
  const float was = started ? *scale : 0.f;
  uint32_t big = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (tid + k * nthr >= nv) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 x = raw[k].quad(q);
      const uint32_t m[4] = {__float_as_uint(x.x) & 0x7FFFFFFFu, __float_as_uint(x.y) & 0x7FFFFFFFu,
                             __float_as_uint(x.z) & 0x7FFFFFFFu, __float_as_uint(x.w) & 0x7FFFFFFFu};
#pragma unroll
      for (int e = 0; e < 4; ++e) big = max(big, m[e] < 0x7F800000u ? m[e] : 0u);
    }
  }
  big = __reduce_max_sync(0xffffffffu, big);
  if (W > 1) {  // one block to the CTA: all its threads are here
    if ((tid & 31) == 0) s_max[tid >> 5] = big;
    __syncthreads();
    for (int w = 0; w < W; ++w) big = max(big, s_max[w]);
  } else {
    __syncwarp();  // every lane has read the old scale
  }
  // The block's own scale, raised to a power of two (a block written by other means may have any), 2^120 at most; a NaN
  // leaves it to the rows.
  const uint32_t wb = __float_as_uint(was) & 0x7FFFFFFFu;
  const float least = wb > 0x7F800000u ? 0.f : fminf(__uint_as_float((wb + 0x7FFFFFu) & 0x7F800000u), pow2f(120));
  const float now = fmaxf(least, pow2f(scale_exp(big)));
  if (started && now != was) {
    // another scale than the block had: its codes once more, on the new one
    const float ratio = was / now;
    uint4* old = reinterpret_cast<uint4*>(a.code[kv] + (unit * a.capacity + lo) * a.hd);
    for (int v = tid; v < static_cast<int>(len - lo) * vpr; v += nthr) {
      const uint4 w = old[v];
      uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 f0 = from_e4m3x2(static_cast<uint16_t>(c[q])), f1 = from_e4m3x2(static_cast<uint16_t>(c[q] >> 16));
        c[q] = to_e4m3x2(f0.x * ratio, f0.y * ratio) | static_cast<uint32_t>(to_e4m3x2(f1.x * ratio, f1.y * ratio)) << 16;
      }
      old[v] = make_uint4(c[0], c[1], c[2], c[3]);
    }
  }
  const float inv = pow2f(127 - static_cast<int>(__float_as_uint(now) >> 23));
  uint4* code = reinterpret_cast<uint4*>(a.code[kv] + (unit * a.capacity + r0) * a.hd);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int v = tid + k * nthr;
    if (v >= nv) continue;
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 x = raw[k].quad(q);
      o[q] = to_e4m3x2(x.x * inv, x.y * inv) | static_cast<uint32_t>(to_e4m3x2(x.z * inv, x.w * inv)) << 16;
    }
    code[v] = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (tid == 0) {
    *scale = now;
    if (kv == 0 && !started) {
      // a block opened by this call: no attention yet, and the next number
      const int64_t held = (len + (1 << a.block_log2) - 1) >> a.block_log2;
      if (a.weight) a.weight[unit * nblk + blk] = 0.f;
      if (a.ids) a.ids[unit * nblk + blk] = (held ? a.ids[unit * nblk + held - 1] + 1 : 0) + static_cast<int32_t>(blk - held);
    }
  }
}

// ------------------------------------------------------------- attention
struct AttendArgs {
  const float* k_scale;
  const float* v_scale;
  const void* q;
  const int32_t* lens;
  float* part;   // partial slots: [gq][hd] sums
  float2* ml;    // [slot][gq] their references and softmax sums
  float* wpart;  // [unit][tile][sub-block][gq] sums of the tile's weights, or NULL
  float* wref;   // [unit][tile][gq] the maxima they refer to
  int2* span;    // [unit] the first and the last CTA whose share meets it
  float* weight;
  float* out;
  int64_t capacity;
  int B, Hkv, gq, hd, block, tiles_cap;
  int ctas;
  float q_scale;  // log2(e) / sqrt(hd)
  int* status;
};

__host__ __device__ inline int sub_rows(int block) { return block < 32 ? block : 32; }

// Units' tiles stand in one line (sequence, head, tile), and CTA c of n takes a
// contiguous share of it: ragged lengths need no more CTAs than the card runs.
// A unit of nt tiles takes nt + 1 places, the last one empty: starting and
// ending a unit costs a CTA about as much as a tile (8 query heads of 64 columns:
// 0.9 and 0.8 thousand clocks of each warpgroup, and a tile 2.8 of one of the two;
// 48 sequences of 1 to 8192 tokens took 32 us by tiles alone).
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
// Rows of sequence b, within the cache (the joining kernel records a length outside), and their tiles.
__device__ __forceinline__ int rows_of(const AttendArgs& a, int b) {
  return min(max(a.lens[b], 0), static_cast<int>(a.capacity));
}
__device__ __forceinline__ int tiles_of(const AttendArgs& a, int b) { return (rows_of(a, b) + kTile - 1) / kTile; }

__device__ __forceinline__ int places_of(int nt) { return nt ? nt + 1 : 0; }

// By one warp: a place of the line.  `target` turns the line's length into the
// place looked for.  A place is told as its sequence b, the places and the units
// that have rows before b; a place past the end is at b = B.
struct Spot {
  int b, before, units;
};
template <typename F>
__device__ inline int walk_line(const AttendArgs& a, Spot* spot, F target) {
  constexpr int kEach = 2;  // sequences a lane takes at a time
  const int lane = threadIdx.x & 31;
  int n[kEach], at = 0;  // the lane's sequences' places, and those before them
  auto load = [&](int base, int carry) {
    int sum = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int b = base + lane * kEach + k;
      n[k] = b < a.B ? places_of(tiles_of(a, b)) * a.Hkv : 0;
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) sum += n[k];
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    at = carry + inc - sum;
    return carry + __shfl_sync(0xffffffffu, inc, 31);
  };
  int total = 0;
  for (int base = 0; base < a.B; base += 32 * kEach) total = load(base, total);
  const int x = target(total);
  *spot = Spot{a.B, total, 0};
  for (int base = 0, carry = 0; base < a.B; base += 32 * kEach) {
    if (a.B > 32 * kEach) carry = load(base, carry);  // else what was loaded still stands
    int hit_k = -1, hit_at = 0, p = at;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      if (x >= p && x < p + n[k]) {
        hit_k = k;
        hit_at = p;
      }
      p += n[k];
    }
    const unsigned hit = __ballot_sync(0xffffffffu, hit_k >= 0);
    int upto = 32 * kEach;  // of this round, the sequences before the place
    if (hit) {
      const int src = __ffs(hit) - 1;
      upto = src * kEach + __shfl_sync(0xffffffffu, hit_k, src);
      spot->b = base + upto;
      spot->before = __shfl_sync(0xffffffffu, hit_at, src);
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const unsigned some = __ballot_sync(0xffffffffu, n[k] > 0);  // lanes whose k-th sequence has rows
      const int lanes = (upto - k + kEach - 1) / kEach;
      spot->units += a.Hkv * __popc(lanes >= 32 ? some : some & ((1u << lanes) - 1u));
    }
    if (hit) break;
  }
  return total;
}

// One role's position in its CTA's share: tile t of the nt tiles of unit (b, h).
struct Walk {
  int b, h, t, nt, len, ahead;  // ahead: the next sequence's rows, loaded before they are needed
  __device__ __forceinline__ void load(const AttendArgs& a, int rows) {
    len = rows;
    nt = (len + kTile - 1) / kTile;
    ahead = b + 1 < a.B ? rows_of(a, b + 1) : 0;
  }
  // The next tile; only where there is one.
  __device__ __forceinline__ void step(const AttendArgs& a) {
    if (++t < nt) return;
    t = 0;
    if (++h < a.Hkv) return;
    h = 0;
    do {
      ++b;
      load(a, ahead);
    } while (nt == 0);
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float redux_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Offset of byte `c` of row `r` in a tile of 128-byte rows under the 128-byte swizzle.
__device__ __forceinline__ uint32_t swz128(uint32_t r, uint32_t c) {
  return r * 128u + ((((c >> 4) ^ r) & 7u) << 4) + (c & 15u);
}

// The small operands as several e4m3 ones.
// Queries: x = sum_i 16^-i piece_i.  A piece holds four significant bits and
// leaves a remainder of at most 2^-4 of itself, exact in f32, as long as it does
// not run out of exponents at 2^-6: two pieces hold bf16 numbers down to 2^-14
// of the head's largest entry, four down to 2^-22 and all to 2^-30 of it (queries
// have columns far above the others, and the keys may make little of them); six
// keep f32 numbers to 2^-38.  Four pieces of four heads are one MMA width, 16.
// Probabilities (times the value scale): fixed point against the tile's largest,
// 32 bits in eight digits of four.  The codes 0 .. 15 of e4m3 stand for 0 .. 15
// times 2^-9 (its subnormals and first binade), so a digit is its own code.  The
// widest tile, whose O of eight columns a head would not fit TMEM, has six pieces
// as the queries have: all 24 bits of a product down to 2^-14 of the tile's largest
// and the rest to 2^-38 of it, where six digits would end at 2^-24 (an attention
// sink, or one large value of a block, leaves the other rows of a tile that far
// below).  They cost the conversions there and back.
template <int GQ, int HDA>
__host__ __device__ constexpr int digits() { return GQ * HDA == 32 ? 6 : 8; }

// Four digits as four bytes: of bytes i and j of a.
__device__ __forceinline__ uint32_t spread(uint32_t a, int i, int j) {
  const uint32_t y = __byte_perm(a, 0u, 0x4040u | i | j << 8);
  return (y | y << 4) & 0x0F0F0F0Fu;
}

// The next piece of two numbers as two codes, and what is left of them times 16.
__device__ __forceinline__ uint32_t next_piece(float& a, float& b, bool last) {
  const uint16_t c = to_e4m3x2(a, b);
  if (!last) {
    const __half2 k16 = __half2half2(__ushort_as_half(0xCC00));  // -16: exact, 448 * 16 fits
    const float2 f = __half22float2(__hmul2(__half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)), k16));
    a = fmaf(a, 16.f, f.x);
    b = fmaf(b, 16.f, f.y);
  }
  return c;
}
template <typename T>
struct Pieces;
template <>
struct Pieces<__nv_bfloat16> {
  static constexpr int n = 4;
  using raw = uint2;  // four elements
  __device__ static __forceinline__ void open(uint2 w, float* v) {
    const float2 a = bf2_to_f2(w.x), b = bf2_to_f2(w.y);
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  }
};
template <>
struct Pieces<float> {
  static constexpr int n = 6;
  using raw = float4;
  __device__ static __forceinline__ void open(float4 w, float* v) {
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
  }
};

// warps 0-7: softmax, two warpgroups taking tiles in turn
constexpr int kWarpTma = 8, kWarpS = 9, kWarpO = 10, kWarpQ = 11, kAttendThreads = 384;
constexpr int kMaxStages = 8;
constexpr int kAtom = kTile * 128;  // bytes of 128 rows x 128 columns

template <typename T, int GQ, int HDA>
struct AttendShape {
  static constexpr int nq = Pieces<T>::n * GQ, np = digits<GQ, HDA>() * GQ;  // operand rows in use
  static constexpr int ns = (nq + 15) / 16 * 16, no = np;                // and MMA widths
  static constexpr int bytes_p = 2 * no * 128;
  static constexpr int cols(int ahead) { return ahead * ns + 2 * HDA * no; }
  static constexpr int stages_of(int ahead) {
    const int s = (227 * 1024 - 9216 - 1024 - bytes_p - ahead * HDA * ns * 128) / (2 * HDA * kAtom);
    return s < kMaxStages ? s : kMaxStages;
  }
  // S runs up to `ahead` tiles before O, in as many buffers of TMEM and of the
  // queries' pieces.
  static constexpr int ahead = cols(4) <= 512 && stages_of(4) >= 3   ? 4
                               : cols(3) <= 512 && stages_of(3) >= 2 ? 3
                               : cols(2) <= 512                      ? 2
                                                                     : 1;
  static constexpr int stages = stages_of(ahead);
  static constexpr int tmem = cols(ahead) <= 64 ? 64 : cols(ahead) <= 128 ? 128 : cols(ahead) <= 256 ? 256 : 512;
  static constexpr int bytes_q = ahead * HDA * ns * 128;
  static_assert(cols(ahead) <= 512 && stages >= 2, "attention pipeline");
  static constexpr int smem = stages * 2 * HDA * kAtom + bytes_p + bytes_q + 1024;
};

// Exact 2^x of a whole x <= 127; 0 below 2^-126.
__device__ __forceinline__ float pow2_whole(float x) {
  const int b = __float_as_int(fmaxf(x, -127.f) + 12582912.f);  // 1.5 * 2^23: x in the low bits
  return __int_as_float((b << 23) + 0x3F800000);
}

// Sums each of p[0..GQ) over groups of `sub` (8, 16 or 32) lanes, halving the
// values a lane holds at each of the first steps; f(g, sum) is called by one
// lane of the group for each g.
template <int GQ, typename F>
__device__ __forceinline__ void group_sums(const float* p, int sub, F f) {
  const int lane = threadIdx.x & 31;
  float v[GQ];
#pragma unroll
  for (int g = 0; g < GQ; ++g) v[g] = p[g];
  int first = 0;
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    const int o = 1 << s, n = GQ >> (s + 1);  // values kept by a lane after the step
    const bool up = lane & o;
    if (n >= 1) {
#pragma unroll
      for (int g = 0; g < n; ++g) {
        const float send = up ? v[g] : v[g + n], keep = up ? v[g + n] : v[g];
        v[g] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
      first += up ? n : 0;
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
  constexpr int kLeft = GQ >= 8 ? GQ / 8 : 1;
#pragma unroll
  for (int o = 8; o < 32; o <<= 1)
    if (o < sub) {
#pragma unroll
      for (int g = 0; g < kLeft; ++g) v[g] += __shfl_xor_sync(0xffffffffu, v[g], o);
    }
  const int who = lane & (sub - 1);
  if (GQ >= 8 ? who < 8 : who < 4) {
#pragma unroll
    for (int g = 0; g < kLeft; ++g) f(first + g, v[g]);
  }
}

// Decode attention on the tensor cores.  For a tile of 128 token rows
//   S = K Q^T   (128 rows x pieces of the group's queries, K = head_dim),
//   O = V^T P^T (128 columns x digits of the probabilities, K = 128 rows):
// the codes go from HBM to the MMA as they are (TMA, 128-byte swizzle), nothing
// is unpacked, and the small operands carry their precision in e4m3 pieces
// instead.  A block's scale enters as a factor of S's row or of P's column.
//   warps 0-3, 4-7: softmax of tiles in turn; thread = token row of S, then
//                   column of O, which is summed in f32 registers;
//   warp 8: TMA of the K and V rings; warps 9, 10: the MMAs of S and of O, of
//   their own so that neither waits for the other's operands; warp 11: the
//   pieces of the next units' queries.
// Rows behind the sequence's end are masked in S, and their V rows zeroed before
// the MMA (0 * NaN).
// Bound by HBM where units are long: 4 sequences of 64K tokens, 8 KV heads of 128
// with 4 query heads each, take 90 us with the join, 6.0 TB/s (537 MB, all of them
// read once: 537.3 MB of DRAM reads; the tensor pipe is 6.6 % busy).  Otherwise by
// the chain of a tile's steps, 2600 to 2850 clocks with 8 query heads, of which two
// warpgroups have one each in flight, and which waits for S for 160 to 220 of them:
// two sequences of 128K tokens, 4 x 7 heads, take 51 us (268 MB), 41 of them 28
// tiles of each warpgroup; 48 sequences of 1 to 8192 tokens, 4 x 8 heads of 64, take
// 23 us (23 MB), where a CTA of eleven tiles runs for 13 us and the slowest, of six
// short units, for 18.  Three warpgroups (512 threads, registers moved to them)
// spilled: 72 us instead of 53 for the two long sequences.
// Registers: 8 query heads of 256 columns and 16 of either width are at the limit of
// 168 a thread and spill 36 to 84 bytes.
template <typename T, int GQ, int HDA>
__global__ void __launch_bounds__(kAttendThreads, 1)
kv8_attend_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const AttendArgs a) {
  using Sh = AttendShape<T, GQ, HDA>;
  constexpr int kStages = Sh::stages, kAhead = Sh::ahead, kNq = Pieces<T>::n;
  // Barriers of a full S.  A warpgroup waits for every other tile, and by parity: when it waits for tile i, the same
  // barrier's use before must have ended.  Tile i - 2, its own, tells it that, with two barriers or more, S being in
  // order; with one, tile i - 1 would still be running, and tile i - 2's phase be taken for tile i's.
  constexpr int kFull = kAhead < 2 ? 2 : kAhead;
  static_assert(kFull >= 2 && kFull % kAhead == 0, "barriers of S");
  constexpr int kDigits = digits<GQ, HDA>();
  constexpr float kUnit = kDigits == 8 ? 4294967296.f : 256.f;  // the digits', or the first piece's, of a tile's 1
  constexpr uint32_t kColO = kAhead * Sh::ns;  // O's first TMEM column, after the buffers of S
  extern __shared__ uint8_t sm_raw[];
  __shared__ __align__(8) uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  __shared__ __align__(8) uint64_t s_full[kFull], s_empty[kAhead], q_full[kAhead], q_empty[kAhead], p_full[2], o_full[2], done[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_tiles[2];
  __shared__ Walk s_walk;
  __shared__ __align__(16) float s_max[2][2][2 * GQ][4];
  __shared__ __align__(16) float4 s_ref[2][2][4][GQ];
  // factors of the logits of the last units: the queries run at most kAhead units before S, S kAhead tiles before P
  constexpr int kFactors = 16;
  static_assert(2 * kAhead + 2 <= kFactors, "factors kept");
  __shared__ float s_qc[kFactors][GQ], s_sum[2][2][4][GQ];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sk = sm;
  uint8_t* sv = sk + kStages * HDA * kAtom;
  uint8_t* sp = sv + kStages * HDA * kAtom;
  uint8_t* sq = sp + Sh::bytes_p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (warp == kWarpO) {  // while warp 0 finds the share
    if (lane < kStages) {
      mbar_init(&k_full[lane], 1);
      mbar_init(&k_empty[lane], 1);
      mbar_init(&v_full[lane], 1);
      mbar_init(&v_empty[lane], 1);
    }
    if (lane < kFull) mbar_init(&s_full[lane], 2);
    if (lane < kAhead) {
      mbar_init(&s_empty[lane], 4);
      mbar_init(&q_full[lane], 32);
      mbar_init(&q_empty[lane], 1);
    }
    if (lane < 2) {
      mbar_init(&p_full[lane], 128);
      mbar_init(&o_full[lane], 1);
      mbar_init(&done[lane], 1);
    }
    if (lane == 0) s_abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarpTma && lane == 0) {
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  wait_for_earlier();
  let_next_start();  // not before: the joining kernel reads the lengths at once
  // nor TMEM, which an earlier kernel on this SM may still ask for while this one waits for it
  if (warp == kWarpS) tmem_alloc(&s_tmem, Sh::tmem);
  if (warp < 2) {  // the share's start by warp 0, its end by warp 1
    Spot spot;
    Share share{0, 0};
    walk_line(a, &spot, [&](int total) {
      share = share_of(total, a.ctas, blockIdx.x);
      return warp ? share.hi : share.lo;
    });
    if (lane == 0) {
      int ended = 0, places = 0;  // units that end before the place
      if (share.lo < share.hi) {
        Walk w;
        w.b = spot.b;
        if (warp == 0) {
          w.load(a, rows_of(a, w.b));
          w.h = (share.lo - spot.before) / (w.nt + 1);
          w.t = share.lo - spot.before - w.h * (w.nt + 1);
          ended = spot.units + w.h;
          places = share.hi - share.lo;
          if (w.t == w.nt && places > 1) {  // the share starts with an empty place
            w.t = w.nt - 1;
            w.step(a);
          }
          s_walk = w;
        } else {
          ended = spot.units;
          if (spot.b < a.B) ended += (share.hi - spot.before) / places_of(tiles_of(a, spot.b));
        }
      }
      // the share's tiles: its places less the empty one of every unit that ends in it
      s_tiles[warp] = places - (warp ? ended : -ended);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int n = s_tiles[0] + s_tiles[1];
  // A wait that runs out sets s_abort, after which no wait waits: the TMA and MMA
  // warps stop, the others run through their loops and meet every barrier.
  volatile int* abort = &s_abort;
  auto wait_one = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (mbar_wait(bar, parity, a.status)) return true;
    *abort = 1;
    return false;
  };
  // By a whole warp, which goes on together, and with one answer.
  auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait_one(bar, parity)) != 0; };
  // By one warp, one, two or four query heads at a time, 32, 16 or 8 lanes to a head: their pieces into the unit's
  // buffer, K-major rows piece * GQ + g, zero past head_dim and past the group, and the factor of their logits.  A lane
  // has four columns of every 4 kLanes, kVecs times; what it does is a chain of short steps, and these run side by side.
  using QRaw = typename Pieces<T>::raw;
  auto query_load = [&](int64_t unit, int g0, auto& raw) {
    constexpr int kVecs = std::extent_v<std::remove_reference_t<decltype(raw)>>, kLanes = 32 * HDA / kVecs;
    constexpr int kStep = 4 * kLanes;  // columns
    const int q_head = lane / kLanes, q_col = 4 * (lane % kLanes);
    const T* q = static_cast<const T*>(a.q) + (unit * a.gq + g0 + q_head) * a.hd;
#pragma unroll
    for (int x = 0; x < kVecs; ++x) {
      const int j = kStep * x + q_col;
      raw[x] = QRaw{};
      if (g0 + q_head < a.gq && j < a.hd) raw[x] = *reinterpret_cast<const QRaw*>(q + j);
    }
  };
  auto query_store = [&](const auto& raw, int g0, int seg) {
    constexpr int kVecs = std::extent_v<std::remove_reference_t<decltype(raw)>>, kLanes = 32 * HDA / kVecs;
    constexpr int kStep = 4 * kLanes;  // columns
    const int q_head = lane / kLanes, q_col = 4 * (lane % kLanes);
    float v[kVecs][4];
    uint32_t big = 0;
#pragma unroll
    for (int x = 0; x < kVecs; ++x) {
      Pieces<T>::open(raw[x], v[x]);
#pragma unroll
      for (int e = 0; e < 4; ++e) big = max(big, __float_as_uint(v[x][e]) & 0x7FFFFFFFu);
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
    const int e2 = scale_exp(big);
    // a head with an entry that is not finite has NaN logits
    const float inv = big < 0x7F800000u ? pow2f(-e2) : __uint_as_float(0x7FC00000u);
    if (lane % kLanes == 0) s_qc[seg % kFactors][g0 + q_head] = pow2f(min(e2, 120)) * a.q_scale;
#pragma unroll
    for (int x = 0; x < kVecs; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[x][e] *= inv;
    // row p * GQ + g0 + q_head, column kStep x + q_col: the swizzle's exclusive or splits into the lane's part and the
    // step's, GQ being 4 or a multiple of 8
    const int row = g0 + q_head;
    uint8_t* to = sq + (seg % kAhead) * HDA * Sh::ns * 128 + row * 128;
    const uint32_t mine = swz128(row, q_col) - row * 128;
#pragma unroll
    for (int p = 0; p < kNq; ++p)
#pragma unroll
      for (int x = 0; x < kVecs; ++x) {
        float* r = v[x];
        const uint32_t c0 = next_piece(r[0], r[1], p + 1 == kNq), c1 = next_piece(r[2], r[3], p + 1 == kNq);
        const uint32_t step = (kStep * x % 128 / 16 ^ ((p * GQ) & 7)) << 4;
        *reinterpret_cast<uint32_t*>(to + (kStep * x / 128) * Sh::ns * 128 + p * GQ * 128 + (mine ^ step)) = c0 | c1 << 16;
      }
  };
  if (n > 0) {
    Walk w = s_walk;
    if (warp == kWarpTma) {
      if (lane == 0) {
        int i = 0;
        for (; i < n; ++i) {
          const int st = i % kStages;
          const uint32_t ph = ((i / kStages) & 1) ^ 1;
          const int unit = w.b * a.Hkv + w.h;
          if (i >= kStages && !wait_one(&k_empty[st], ph)) break;
          mbar_arrive_expect_tx(&k_full[st], HDA * kAtom);
          for (int x = 0; x < HDA; ++x)
            tma_load_3d(sk + (st * HDA + x) * kAtom, &map_k, &k_full[st], 128 * x, w.t * kTile, unit);
          if (i >= kStages && !wait_one(&v_empty[st], ph)) {
            drain_ring(k_full, kStages, i + 1, a.status);
            drain_ring(v_full, kStages, i, a.status);
            i = -1;
            break;
          }
          mbar_arrive_expect_tx(&v_full[st], HDA * kAtom);
          for (int x = 0; x < HDA; ++x)
            tma_load_3d(sv + (st * HDA + x) * kAtom, &map_v, &v_full[st], 128 * x, w.t * kTile, unit);
          if (i + 1 < n) w.step(a);
        }
        if (i >= 0 && i < n) {
          drain_ring(k_full, kStages, i, a.status);
          drain_ring(v_full, kStages, i, a.status);
        }
      }
    } else if (warp == kWarpS) {
      // S of tile i, once its K is there and tile i - kAhead has been read out of its buffer
      constexpr uint32_t id_s = umma_idesc_e4m3(128, Sh::ns);
      const uint64_t dk = umma_desc_sw128(smem_u32(sk)), dq = umma_desc_sw128(smem_u32(sq));
      const int ksteps = (a.hd + 31) / 32;
      int st = 0, sb = 0, qb = 0;
      uint32_t kph = 0, qph = 0, sph = 1;
      for (int i = 0; i < n; ++i) {
        if (i >= kAhead && !wait(&s_empty[sb], sph)) break;
        if ((i == 0 || w.t == 0) && !wait(&q_full[qb], qph)) break;
        if (!wait(&k_full[st], kph)) break;
        const bool ends = w.t == w.nt - 1 || i == n - 1;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t ka = dk + st * (HDA * kAtom >> 4), qa = dq + qb * (HDA * Sh::ns * 128 >> 4);
#pragma unroll
          for (int k = 0; k < 4 * HDA; ++k)
            if (k < ksteps)
              umma_e4m3(tmem + sb * Sh::ns, ka + (k / 4) * (kAtom >> 4) + (k % 4) * 2,
                        qa + (k / 4) * (Sh::ns * 128 >> 4) + (k % 4) * 2, id_s, k > 0);
          umma_commit(&s_full[i % kFull]);
          mbar_arrive(&s_full[i % kFull]);  // hands on the factors, which this warp saw with the queries
          umma_commit(&k_empty[st]);
          if (ends) umma_commit(&q_empty[qb]);
        }
        __syncwarp();
        if (++st == kStages) {
          st = 0;
          kph ^= 1;
        }
        if (++sb == kAhead) {
          sb = 0;
          sph ^= 1;
        }
        if (ends && ++qb == kAhead) {
          qb = 0;
          qph ^= 1;
        }
        if (i + 1 < n) w.step(a);
      }
      if (elect_one()) umma_commit(&done[0]);  // what was issued ends before the CTA's memory goes
      (void)mbar_wait(&done[0], 0, a.status);
    } else if (warp == kWarpO) {
      constexpr uint32_t id_o = umma_idesc_e4m3(128, Sh::no, true, true);
      const uint64_t dv = umma_desc_sw128_mn(smem_u32(sv), kAtom, 1024), dp = umma_desc_sw32_mn(smem_u32(sp), kTile * 32, 256);
      int st = 0;
      uint32_t vph = 0;
      for (int i = 0; i < n; ++i) {
        const int wg = i & 1;
        if (!wait(&v_full[st], vph) || !wait(&p_full[wg], (i >> 1) & 1)) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t va = dv + st * (HDA * kAtom >> 4), pa = dp + wg * (Sh::no * 128 >> 4);
#pragma unroll
          for (int x = 0; x < HDA; ++x)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_e4m3(tmem + kColO + (wg * HDA + x) * Sh::no, va + x * (kAtom >> 4) + k * (4096 >> 4), pa + k * (1024 >> 4),
                        id_o, k > 0);
          umma_commit(&o_full[wg]);
          umma_commit(&v_empty[st]);
        }
        __syncwarp();
        if (++st == kStages) {
          st = 0;
          vph ^= 1;
        }
      }
      if (elect_one()) umma_commit(&done[1]);
      (void)mbar_wait(&done[1], 0, a.status);
    } else if (warp == kWarpQ) {
      // the queries of every unit after the first, as far ahead as there are buffers; the next unit's are loaded
      // (32 registers of them at most) while one is cut into pieces
      constexpr int kQuads = 4 * HDA;  // eight lanes to a head
      constexpr int kMost = 128 / (kQuads * static_cast<int>(sizeof(QRaw)));
      constexpr int kBatch = kMost < GQ / 4 ? kMost : GQ / 4;
      QRaw raw[kBatch][kQuads], next[kBatch][kQuads];
      int64_t unit = 0;
      int seg = -1;
      for (int i = 0; seg < 0 || unit >= 0; ++seg) {
        // the unit after this one
        i += w.nt - w.t;
        int64_t after = -1;
        if (i < n) {
          w.t = w.nt - 1;
          w.step(a);
          after = static_cast<int64_t>(w.b) * a.Hkv + w.h;
#pragma unroll
          for (int k = 0; k < kBatch; ++k) query_load(after, 4 * k, next[k]);
        }
        if (seg >= 0) {
          const int s1 = seg + 1, qb = s1 % kAhead;
          if (s1 >= kAhead) (void)wait(&q_empty[qb], ((s1 / kAhead) & 1) ^ 1);
#pragma unroll 1
          for (int g0 = 0; g0 < GQ; g0 += 4 * kBatch) {
            if (g0 > 0)
#pragma unroll
              for (int k = 0; k < kBatch; ++k) query_load(unit, g0 + 4 * k, raw[k]);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) query_store(raw[k], g0 + 4 * k, s1);
          }
          fence_proxy_async();
          mbar_arrive(&q_full[qb]);
        }
        unit = after;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
#pragma unroll
          for (int x = 0; x < kQuads; ++x) raw[k][x] = next[k][x];
      }
    } else {
      // the first unit's queries, which everything waits for, by a softmax warp for each head, or for every two
      constexpr int kHeadsEach = GQ > 8 ? 2 : 1;
      if (warp * kHeadsEach < GQ) {
        QRaw raw[kHeadsEach * HDA];
        query_load(static_cast<int64_t>(w.b) * a.Hkv + w.h, kHeadsEach * warp, raw);
        query_store(raw, kHeadsEach * warp, 0);
      }
      fence_proxy_async();
      named_bar_sync(3, 256);
      if (warp == 0) mbar_arrive(&q_full[0]);
      const int wg = warp >> 2, row = tid & 127, quarter = warp & 3;
      const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
      const int lb = 31 - __clz(a.block), sub = sub_rows(a.block), ls = min(lb, 5), spt = kTile >> ls;
      const int64_t nblk = a.capacity >> lb;
      // this token's row of P: 32 bytes in each block of 32 digits, 16-byte halves swapped by the 32-byte swizzle
      uint8_t* p_row = sp + wg * Sh::no * 128 + row * 32;
      const int p_flip = (row & 4) << 2;
      float acc[HDA][GQ], l[GQ], c[GQ];
      float m = -INFINITY;  // lane g: the running reference of head g, a whole number
      // O of use `u` (the u-th tile of this warpgroup) into the sums
      auto fold = [&](int u) {
        (void)wait(&o_full[wg], u & 1);
        tc_fence_after();
        const float4* ref = s_ref[wg][u & 1][quarter];
#pragma unroll
        for (int x = 0; x < HDA; ++x) {
          float sum[GQ];
#pragma unroll
          for (int g = 0; g < GQ; ++g) sum[g] = 0.f;
          constexpr int kHeads = kDigits == 8 ? 4 : 8, kCols = kHeads * kDigits;  // heads read at a time
#pragma unroll
          for (int g0 = 0; g0 < GQ; g0 += kHeads) {
            float v[kCols];
#pragma unroll
            for (int k = 0; k < kCols; k += 16)
              tmem_ld16(tmem + lanes + kColO + (wg * HDA + x) * Sh::no + g0 * kDigits + k, v + k);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < kCols; ++k) sum[g0 + k / kDigits] = fmaf(sum[g0 + k / kDigits], 0.0625f, v[k]);
          }
#pragma unroll
          for (int g = 0; g < GQ; ++g) {
            const float2 r = *reinterpret_cast<const float2*>(&ref[g].z);
            acc[x][g] = fmaf(sum[g], r.y, acc[x][g] * r.x);
          }
        }
      };
      int seg = 0;
      for (int i0 = 0; i0 < n; ++seg) {
        // one unit: tiles i0 .. i1 - 1 of the share, t0 ... of the unit; this warpgroup's are every other one
        const int64_t unit = static_cast<int64_t>(w.b) * a.Hkv + w.h;
        const int t0 = w.t, i1 = min(n, i0 + w.nt - t0);
        const int first = i0 + ((i0 ^ wg) & 1);
        if (tid == 0) {
          if (t0 == 0) a.span[unit].x = blockIdx.x;
          if (t0 + i1 - i0 == w.nt) a.span[unit].y = blockIdx.x;
        }
        const int len = w.len;
        const float* ksp = a.k_scale + unit * nblk;
        const float* vsp = a.v_scale + unit * nblk;
        float* wp = a.wpart ? a.wpart + unit * a.tiles_cap * spt * a.gq : nullptr;
        float* wr = a.wref + unit * a.tiles_cap * a.gq;
        int at = (t0 + first - i0) * kTile + row;
        // scales of the warpgroup's tiles, loaded two of them ahead
        float ks = 1.f, vs = 1.f, ks1 = 1.f, vs1 = 1.f;  // 1 for rows past the end
        auto scales = [&](int k, float* x, float* y) {
          const int r = at + k * 2 * kTile;
          if (first + 2 * k < i1 && r < len) {
            *x = ksp[r >> lb];
            *y = vsp[r >> lb];
          }
        };
        scales(0, &ks, &vs);
        scales(1, &ks1, &vs1);
#pragma unroll
        for (int g = 0; g < GQ; ++g) {
          l[g] = 0.f;
#pragma unroll
          for (int x = 0; x < HDA; ++x) acc[x][g] = 0.f;
        }
        m = -INFINITY;
        for (int i = first; i < i1; i += 2, at += 2 * kTile) {
          const int use = i >> 1, par = use & 1, sb = i % kAhead, t = t0 + i - i0;
          const bool live = at < len;
          (void)wait(&s_full[i % kFull], (i / kFull) & 1);
          tc_fence_after();
          if (i == first) {
#pragma unroll
            for (int g = 0; g < GQ; ++g) c[g] = s_qc[seg % kFactors][g];
          }
          float ks2 = 1.f, vs2 = 1.f;
          if (i + 4 < i1 && at + 4 * kTile < len) {
            ks2 = ksp[(at + 4 * kTile) >> lb];
            vs2 = vsp[(at + 4 * kTile) >> lb];
          }
          float s[GQ];
#pragma unroll
          for (int g = 0; g < GQ; ++g) s[g] = 0.f;
          constexpr int kCols = Sh::ns <= 48 ? Sh::ns : 48;
#pragma unroll
          for (int k0 = (Sh::ns - 1) / kCols * kCols; k0 >= 0; k0 -= kCols) {
            float v[kCols];
#pragma unroll
            for (int k = 0; k < kCols; k += 16) tmem_ld16(tmem + lanes + sb * Sh::ns + k0 + k, v + k);
            tmem_ld_wait();
#pragma unroll
            for (int k = kCols - 1; k >= 0; --k)
              if (k0 + k < Sh::nq) s[(k0 + k) % GQ] = fmaf(s[(k0 + k) % GQ], 0.0625f, v[k]);
          }
          tc_fence_before();
          if (lane == 0) mbar_arrive(&s_empty[sb]);
          // The tile's largest logits, and the largest of logit + log2(value scale), which is what a row brings to
          // O: references are whole numbers, so that every change of one is an exact power of two.
          const uint32_t vb = __float_as_uint(vs), frac = vb & 0x7FFFFFu;  // vs = vm 2^ev, vm in (1/2, 1]
          const float ev = static_cast<float>(static_cast<int>(vb >> 23) - 127 + (frac ? 1 : 0));
          const float vm = __uint_as_float(frac | (frac ? 0x3F000000u : 0x3F800000u)) * kUnit;
#pragma unroll
          for (int g = 0; g < GQ; ++g) s[g] = live ? s[g] : -INFINITY;  // times a positive factor
          if (lb >= 5) {  // a warp's rows share a scale, its first row's
#pragma unroll
            for (int g = 0; g < GQ; ++g) {
              const float x0 = redux_max(s[g] * (c[g] * ks));
              if (lane == 0) {
                s_max[wg][par][2 * g][quarter] = x0;
                s_max[wg][par][2 * g + 1][quarter] = x0 + ev;
              }
            }
          } else {
#pragma unroll
            for (int g = 0; g < GQ; ++g) {
              const float x = s[g] * (c[g] * ks);
              const float x0 = redux_max(x), x1 = redux_max(x + ev);
              if (lane == 0) {
                s_max[wg][par][2 * g][quarter] = x0;
                s_max[wg][par][2 * g + 1][quarter] = x1;
              }
            }
          }
          named_bar_sync(1 + wg, 128);
          float4* ref = s_ref[wg][par][quarter];  // {reference, -reference of O, factors of the sums and of O}
          if (lane < GQ) {
            const float4 x0 = *reinterpret_cast<const float4*>(s_max[wg][par][2 * lane]);
            const float4 x1 = *reinterpret_cast<const float4*>(s_max[wg][par][2 * lane + 1]);
            const float mn = fmaxf(m, ceilf(fmaxf(fmaxf(x0.x, x0.y), fmaxf(x0.z, x0.w))));
            const float mv = ceilf(fmaxf(fmaxf(x1.x, x1.y), fmaxf(x1.z, x1.w)));
            const float al = m == mn ? 1.f : pow2_whole(m - mn);
            // O's digits are 2^-9 of what they stand for, its sum is in units of the highest, 1 is 16 of those; of
            // pieces, it is in units of the first
            ref[lane] = make_float4(mn, mv, al, ex2(mv - mn) * (kDigits == 8 ? 512.f / 16.f : 1.f / kUnit));
            m = mn;
          }
          if (use > 0 && i > first) fold(use - 1);
          __syncwarp();
          float p[GQ], pv[GQ];
#pragma unroll
          for (int g = 0; g < GQ; ++g) {
            const float4 r = ref[g];
            const float ck = c[g] * ks;
            p[g] = ex2(fmaf(s[g], ck, -r.x));
            l[g] = fmaf(l[g], r.z, p[g]);
            pv[g] = ex2(fmaf(s[g], ck, ev - r.y)) * vm;
          }
          auto put = [&](int k, const uint32_t* o) {  // sixteen columns of this token's row
            *reinterpret_cast<uint4*>(p_row + (k / 2) * kTile * 32 + (((k & 1) * 16) ^ p_flip)) =
                make_uint4(o[0], o[1], o[2], o[3]);
          };
          if constexpr (kDigits == 8) {
#pragma unroll
            for (int k = 0; k < Sh::no / 16; ++k) {
              uint32_t o[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                // a NaN is 0 here, and the sum l has it; 1 itself is the largest number below it
                const uint32_t fix = __float2uint_rn(pv[2 * k + e / 2]);
                o[e] = spread(fix, 2 * (e & 1), 2 * (e & 1) + 1);
              }
              put(k, o);
            }
          } else {
            // the last piece first, as the digits' lowest: twelve bytes of two heads, 48 of eight
#pragma unroll
            for (int g0 = 0; g0 < GQ; g0 += 8) {
              uint32_t o[12];
#pragma unroll
              for (int g = 0; g < 8; g += 2) {
                uint32_t c2[3];  // two pieces of both heads, from the first ones
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                  const uint32_t a0 = next_piece(pv[g0 + g], pv[g0 + g + 1], false);
                  c2[x] = a0 << 16 | next_piece(pv[g0 + g], pv[g0 + g + 1], x == 2);
                }
                o[g / 2 * 3] = __byte_perm(c2[2], c2[1], 0x6420);
                o[g / 2 * 3 + 1] = __byte_perm(c2[0], c2[2], 0x7520);
                o[g / 2 * 3 + 2] = __byte_perm(c2[1], c2[0], 0x7531);
              }
#pragma unroll
              for (int k = 0; k < 3; ++k) put(g0 / 8 * 3 + k, o + 4 * k);
            }
          }
          if (len - t * kTile < kTile) {
            const int st = i % kStages;
            (void)wait(&v_full[st], (i / kStages) & 1);
            if (!live) {
#pragma unroll
              for (int x = 0; x < HDA; ++x)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  reinterpret_cast<uint4*>(sv + (st * HDA + x) * kAtom + row * 128)[k] = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async();
          tc_fence_before();
          mbar_arrive(&p_full[wg]);
          if (wp) {
            float* wt = wp + (static_cast<int64_t>(t) * spt + (row >> ls)) * a.gq;
            group_sums<GQ>(p, sub, [&](int g, float sum) {
              if (g < a.gq) wt[g] = sum;
            });
            if (quarter == 0 && lane < a.gq) wr[static_cast<int64_t>(t) * a.gq + lane] = m;
          }
          ks = ks1;
          vs = vs1;
          ks1 = ks2;
          vs1 = vs2;
        }
        if (first < i1) {
          // the unit's partial of this warpgroup
          fold(((i1 - 1 - wg) & ~1) / 2);
          float* slot = a.part + (2 * (unit + blockIdx.x) + wg) * (a.gq * a.hd);
#pragma unroll
          for (int g = 0; g < GQ; ++g)
#pragma unroll
            for (int x = 0; x < HDA; ++x)
              if (g < a.gq && row + 128 * x < a.hd) slot[g * a.hd + row + 128 * x] = acc[x][g];
          float(*sums)[GQ] = s_sum[wg][seg & 1];  // read before the warpgroup's barrier after next
          group_sums<GQ>(l, 32, [&](int g, float sum) { sums[quarter][g] = sum; });
          named_bar_sync(1 + wg, 128);
          if (row < a.gq)
            a.ml[(2 * (unit + blockIdx.x) + wg) * a.gq + row] =
                make_float2(m, (sums[0][row] + sums[1][row]) + (sums[2][row] + sums[3][row]));
        } else if (row < a.gq) {  // no tile of the unit: a slot that weighs nothing
          a.ml[(2 * (unit + blockIdx.x) + wg) * a.gq + row] = make_float2(-INFINITY, 0.f);
        }
        // to the next unit
        i0 = i1;
        if (i0 < n) {
          w.t = w.nt - 1;
          w.step(a);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpS) tmem_dealloc(tmem, Sh::tmem);
}

// Joins a unit's partials: out = sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i.
// CTA (unit, y) takes `heads` (1, 2, 4 or 8) query heads, each by 8 / heads warps,
// a warp by slot; CTAs (unit, y >= head_ctas) add a share of the blocks' weights,
// sum_g 2^(ref - M_g) wpart / L_g.  What it costs is latency, so every thread has
// its loads in flight together, one CTA takes several heads where there are
// units enough, and the launch is a programmatic one.  Which CTAs met the unit is
// read as the attention wrote it: found again from the lengths, while the attention
// ran, it cost 1.1 us for 8 heads, beside whose 168 registers a thread these CTAs find no
// room before the attention's end (one-tile units: 10.7 -> 9.6 us).  About 2.5 us after the attention's end for two
// sequences of 128K tokens (38 slots to each of 8 x 7 heads, 1024 blocks).
constexpr int kCombineThreads = 256;
constexpr int kMaxSlots = 2 * 256;      // of one unit: two for each CTA
constexpr int kWeightBlocks = 64;       // blocks whose weights a CTA has in hand at a time

__global__ void __launch_bounds__(kCombineThreads, 4) kv8_combine_kernel(const AttendArgs a, int heads, int head_ctas) {
  __shared__ float s_f[8][kMaxSlots];
  __shared__ float s_m[16], s_r[16];
  __shared__ __align__(16) float s_red[8][256];
  const int unit = blockIdx.x, b = unit / a.Hkv, gq = a.gq, hd = a.hd;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  let_next_start();
  // the lengths: the attention kernel lets this one start only when what came before it is done
  const int len = static_cast<int>(checked_len(a.lens[b], a.capacity, a.status));
  const int nt = (len + kTile - 1) / kTile;
  wait_for_earlier();  // what the attention wrote from here on
  int c0 = 0, c1 = 0;  // the CTAs whose shares met the unit
  if (nt) {
    const int2 c = a.span[unit];
    c0 = c.x;
    c1 = c.y;
  }
  float* out = a.out + static_cast<int64_t>(unit) * gq * hd;
  if (nt == 0) {
    if (blockIdx.y == 0)
      for (int i = tid; i < gq * hd; i += kCombineThreads) out[i] = 0.f;
    return;
  }
  // the unit's slots: two for each CTA whose share meets it
  const int sf = gq * hd, slots = 2 * (c1 - c0 + 1);
  const float* base = a.part + 2 * static_cast<int64_t>(unit + c0) * sf;
  // by one warp: head g's largest reference M and 1 / L, and (where `f` is one) every slot's 2^(m - M), NaN for a slot
  // without rows
  auto head = [&](int g, float* f) {
    constexpr int kHeld = 2;  // slots a lane holds: 64 in all, the rest in further rounds
    const float2* ml = a.ml + 2 * static_cast<int64_t>(unit + c0) * gq + g;  // below 2^31 from here on: 512 slots
    float M = -INFINITY, L = 0.f;
    for (int from = 0; from < slots; from += 32 * kHeld) {
      float m[kHeld], l[kHeld];
#pragma unroll
      for (int e = 0; e < kHeld; ++e) {
        const int k = from + 32 * e + lane;
        const float2 x = k < slots ? ml[k * gq] : make_float2(-INFINITY, 0.f);
        m[e] = x.x;
        l[e] = x.y;
      }
      float top = M;
#pragma unroll
      for (int e = 0; e < kHeld; ++e) top = fmaxf(top, m[e]);
      top = warp_max(top);
      if (top != M) L *= exp2f(M - top);
      M = top;
#pragma unroll
      for (int e = 0; e < kHeld; ++e) {
        // a slot without rows has l = 0; m = M = -inf where all of a unit's logits are NaN
        const float w = l[e] == 0.f ? 0.f : m[e] == M ? 1.f : exp2f(m[e] - M);
        L = fmaf(l[e], w, L);  // 0 * NaN too: a slot whose every logit is NaN refers to -inf
        const int k = from + 32 * e + lane;
        if (f && k < slots) f[k] = l[e] == 0.f ? NAN : slots <= 32 * kHeld ? w : m[e];
      }
    }
    if (f && slots > 32 * kHeld)  // M has moved since: from the references again
      for (int k = lane; k < slots; k += 32)
        if (!isnan(f[k])) f[k] = f[k] == M ? 1.f : exp2f(f[k] - M);
    L = warp_sum(L);
    if (lane == 0) {
      s_m[g] = M;
      s_r[g] = 1.f / L;
    }
  };
  if (static_cast<int>(blockIdx.y) < head_ctas) {
    const int wph = 8 / heads, slot = warp / wph, part = warp % wph, g = blockIdx.y * heads + slot;
    // a lane has four columns, and four more 128 columns on; the first slots' sums are loaded before their factors
    // are known
    constexpr int kHeld = 4;
    const float* sums = base + g * hd + 4 * lane;
    const bool lo = 4 * lane < hd, hi = 4 * lane + 128 < hd;
    float4 v[kHeld], z[kHeld];
    auto load = [&](int from) {
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const int k = from + j * wph;
        if (lo && k < slots) v[j] = *reinterpret_cast<const float4*>(sums + k * sf);
        if (hi && k < slots) z[j] = *reinterpret_cast<const float4*>(sums + k * sf + 128);
      }
    };
    if (g < gq) {
      load(part);
      if (part == 0) head(g, s_f[slot]);
    }
    __syncthreads();
    if (g < gq) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      auto add = [](float4& s, float f, const float4& t) {
        s.x = fmaf(f, t.x, s.x);
        s.y = fmaf(f, t.y, s.y);
        s.z = fmaf(f, t.z, s.z);
        s.w = fmaf(f, t.w, s.w);
      };
      for (int from = part; from < slots; from += kHeld * wph) {
        if (from != part) load(from);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
          const int k = from + j * wph;
          const float f = k < slots ? s_f[slot][k] : NAN;
          if (isnan(f)) continue;  // a slot without rows holds anything
          if (f == 0.f) {          // of a slot that weighs nothing, NaN alone: values near f32's largest may sum to inf
            auto nan_only = [](float4& t) {
              t = make_float4(isnan(t.x) ? t.x : 0.f, isnan(t.y) ? t.y : 0.f, isnan(t.z) ? t.z : 0.f, isnan(t.w) ? t.w : 0.f);
            };
            nan_only(v[j]);
            nan_only(z[j]);
          }
          add(x, f, v[j]);
          if (hi) add(y, f, z[j]);
        }
      }
      if (lo) *reinterpret_cast<float4*>(&s_red[warp][4 * lane]) = x;
      if (hi) *reinterpret_cast<float4*>(&s_red[warp][4 * lane + 128]) = y;
    }
    __syncthreads();
    for (int i = tid; i < heads * 256; i += kCombineThreads) {
      const int hh = i >> 8, col = i & 255, gg = blockIdx.y * heads + hh;
      if (gg >= gq || col >= hd) continue;
      float o = 0.f;
      for (int k = 0; k < wph; ++k) o += s_red[hh * wph + k][col];
      out[gg * hd + col] = o * s_r[gg];
    }
    return;
  }
  // sixteen threads (heads) to a block, four blocks a thread; the first blocks' sums are in flight while the heads'
  // own are found
  const int lb = 31 - __clz(a.block), n = (len + a.block - 1) >> lb;
  const int ls = min(lb, 5), spb = 1 << (lb - ls);  // a block's sub-blocks
  const int g = tid & 15;
  const float* ref = a.wref + static_cast<int64_t>(unit) * a.tiles_cap * gq + g;
  const float* p = a.wpart + static_cast<int64_t>(unit) * a.tiles_cap * (kTile >> ls) * gq + g;
  float* weight = a.weight + static_cast<int64_t>(unit) * (a.capacity >> lb);
  float r[4], v[4][4], old[4];
  auto load = [&](int k0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + 16 * j + (tid >> 4);
      const bool in = g < gq && k < n;
      r[j] = in ? ref[(k >> (7 - lb)) * gq] : 0.f;
      old[j] = k < n ? weight[k] : 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[j][e] = in && e < spb ? p[static_cast<int64_t>(k * spb + e) * gq] : 0.f;
    }
  };
  const int first = (blockIdx.y - head_ctas) * kWeightBlocks;
  if (first >= n) return;
  load(first);
  for (int h8 = warp; h8 < gq; h8 += 8) head(h8, nullptr);
  __syncthreads();
  const float mg = g < gq ? s_m[g] : 0.f, rg = g < gq ? s_r[g] : 0.f;
  for (int k0 = first; k0 < n; k0 += (gridDim.y - head_ctas) * kWeightBlocks) {
    if (k0 != first) load(k0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + 16 * j + (tid >> 4);
      float w = g < gq && k < n ? ((v[j][0] + v[j][1]) + (v[j][2] + v[j][3])) * (exp2f(r[j] - mg) * rg) : 0.f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
      if (g == 0 && k < n) weight[k] = old[j] + w;
    }
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
  int ctas;  // of a unit's cluster
  int keys;  // that shared memory has room for
  int group;       // moves of a piece at most
  uint32_t magic;  // v * magic >> 16 is v / vectors of a block, for v < 256 and blocks of up to 128
  int* status;
};
constexpr int kEvictCtas = 8;       // CTAs (one cluster) per unit at most; those of sequences within the budget leave at once
constexpr int kEvictThreads = 256;
constexpr int kEvictHeld = 8;         // keys that a thread holds in registers
constexpr int64_t kEvictKeys = 16384;  // and a CTA in shared memory, three CTAs to an SM: past these they are read again
constexpr int64_t kEvictMaxBlocks = 131072;  // three bit-mask arrays of a unit's blocks in shared memory

// Order of a weight among the evictable blocks as an unsigned number: NaN below
// every number, -0 as 0, and below the protected blocks' 0xFFFFFFFF.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sums of n small counts f(i) into out[], by one warp; returns
// their total.
template <typename F>
__device__ inline int warp_scan(int n, int* out, F f) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  for (int base = 0; base < n; base += 32) {
    const int i = base + lane;
    const int v = i < n ? f(i) : 0;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (i < n) out[i] = carry + inc - v;
    carry += __shfl_sync(0xffffffffu, inc, 31);
  }
  return carry;
}

// Position of the r-th (from 0) set bit of `mask`: one for a whole warp, or a
// lane's own.
__device__ __forceinline__ int nth_bit_warp(uint32_t mask, int r) {
  const int lane = threadIdx.x & 31;
  const bool is = ((mask >> lane) & 1u) && __popc(mask & ((1u << lane) - 1u)) == r;
  return __ffs(__ballot_sync(0xffffffffu, is)) - 1;
}
__device__ __forceinline__ int nth_bit(uint32_t mask, int r) {
  int at = 0;
#pragma unroll
  for (int half = 16; half > 0; half >>= 1) {
    const int c = __popc(mask & ((1u << half) - 1u));
    if (r >= c) {
      r -= c;
      mask >>= half;
      at += half;
    }
  }
  return at;
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
// keys itself (radix selection, eight bits a pass; up to 2048 keys stay in
// registers, up to 16384 in shared memory), then the warps of the cluster move
// the kept blocks that stand past the budget into the slots set free below it.
// Slots read (>= budget - 1) and written (< budget) meet only in slot budget - 1,
// which the last move writes: the warp that moves a piece out of it moves the last
// block's piece in.  kGroups: blocks of 2 KB at most, of which a warp moves several
// at a time.
// Four sequences cut from 16K to 8K tokens, 8 heads of 128 (35 MB to move), take
// 18 us: 5 of selection, a chain of block-wide steps, 8 of moves (9 TB/s read and
// written, the writes into L2) and the rest launch, loads and prefix sums.  Sixty
// units cut from 5113 blocks of 8 x 48 to 2556 (59 MB to move) take 57 us, 178 with
// one move at a time: the selection is 9 of them (that instantiation spills 20
// bytes at its 80 registers, three CTAs an SM).
template <bool kGroups>
__global__ void __launch_bounds__(kEvictThreads, 3) kv8_evict_kernel(const EvictArgs a) {
  extern __shared__ uint32_t s_dyn[];
  __shared__ uint32_t s_hist[2][256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need, s_moves, s_whole;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % a.ctas, unit = blockIdx.x / a.ctas, b = unit / a.Hkv;
  let_next_start();
  wait_for_earlier();
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
  constexpr int kHeld = kEvictHeld, kChunk = kHeld * kEvictThreads;
  const bool held = n <= kChunk;
  const int nw = (n + 31) / 32;
  const int last = ids[n - 1];
  auto key_of = [&](int i, float w, int id) {
    const bool safe = id < a.sink || static_cast<int64_t>(id) > static_cast<int64_t>(last) - a.recent || i == n - 1;
    return safe ? 0xFFFFFFFFu : weight_key(w);
  };
  // keys of slots i, i + 256, ... (0 past the end), their loads in flight together
  auto read = [&](int i, uint32_t* u) {
    float w[kHeld];
    int id[kHeld];
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
      const bool in = i + k * kEvictThreads < n;
      w[k] = in ? weight[i + k * kEvictThreads] : 0.f;
      id[k] = in ? ids[i + k * kEvictThreads] : 0;
    }
#pragma unroll
    for (int k = 0; k < kHeld; ++k) u[k] = i + k * kEvictThreads < n ? key_of(i + k * kEvictThreads, w[k], id[k]) : 0u;
  };
  uint32_t mine[kHeld];
  uint32_t* keys = s_dyn + 3 * nw;  // a thread reads only those that it wrote
  const bool stored = !held && n <= a.keys;
  if (held) {
    read(tid, mine);
  } else if (stored) {
    for (int i = tid; i < n; i += kChunk) {
      read(i, mine);
#pragma unroll
      for (int k = 0; k < kHeld; ++k)
        if (i + k * kEvictThreads < n) keys[i + k * kEvictThreads] = mine[k];
    }
  }
  // f(i, key) for the thread's slots, a warp's together
  auto each = [&](auto f) {
    if (held) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k)
        if (k * kEvictThreads < n) f(tid + k * kEvictThreads, mine[k]);
    } else {
      for (int base = 0; base < n; base += kChunk) {
        if (stored) {
#pragma unroll
          for (int k = 0; k < kHeld; ++k) mine[k] = base + tid + k * kEvictThreads < n ? keys[base + tid + k * kEvictThreads] : 0u;
        } else {
          read(base + tid, mine);
        }
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
          if (base + k * kEvictThreads < n) f(base + tid + k * kEvictThreads, mine[k]);
      }
    }
  };
  // the budget-th largest key
  if (tid == 0) {
    s_prefix = 0;
    s_need = a.budget;
    s_whole = 0;
  }
  s_hist[0][tid] = 0;
  __syncthreads();
  // done early where every key of the last bin is kept: two passes, as a rule, for weights without ties
  for (int pass = 0; pass < 4 && !s_whole; ++pass) {
    const int shift = 24 - 8 * pass;
    uint32_t* hist = s_hist[pass & 1];
    const uint32_t prefix = s_prefix, mask = pass == 0 ? 0u : 0xFFFFFFFFu << (shift + 8);
    each([&](int i, uint32_t u) {
      if (i < n && (u & mask) == prefix) atomicAdd(&hist[(u >> shift) & 255u], 1u);
    });
    __syncthreads();
    s_hist[~pass & 1][tid] = 0;
    if (warp == 0) {
      // lane l holds bins 255 - 8 l .. 248 - 8 l; the first bin, from above, that reaches the need
      uint32_t c[8], sum = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        c[k] = hist[255 - 8 * lane - k];
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
      __syncwarp();
      if (above < need && inc >= need) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (above < need && above + c[k] >= need) {
            s_prefix = prefix | static_cast<uint32_t>(255 - 8 * lane - k) << shift;
            s_need = static_cast<int>(need - above);
            s_whole = need - above == c[k];
            above = 0xFFFFFFFFu;
          } else if (above != 0xFFFFFFFFu) {
            above += c[k];
          }
        }
      }
    }
    __syncthreads();
  }
  // bit masks: keys above the threshold, and of those equal to it the lowest `need`; or, where a bin is kept as a
  // whole, all keys from its first on
  const uint32_t threshold = s_prefix;
  const int need = s_need;
  const bool whole = s_whole;
  uint32_t* keep = s_dyn;
  int* pref_m = reinterpret_cast<int*>(s_dyn + nw);
  uint32_t* equal = s_dyn + 2 * nw;
  each([&](int i, uint32_t u) {
    const unsigned gt = __ballot_sync(0xffffffffu, i < n && (u > threshold || (whole && u == threshold)));
    const unsigned eq = __ballot_sync(0xffffffffu, i < n && u == threshold);
    if (lane == 0 && i < n) {
      keep[i >> 5] = gt;
      equal[i >> 5] = eq;
    }
  });
  // this CTA has read weights and numbers: others may change them once all have
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  __syncthreads();
  if (!whole) {
    if (warp == 0) warp_scan(nw, pref_m, [&](int w) { return __popc(equal[w]); });
    __syncthreads();
    for (int w = tid; w < nw; w += kEvictThreads) {
      int take = need - pref_m[w];
      uint32_t eq = equal[w], add = 0;
      while (take > 0 && eq) {
        add |= eq & (0u - eq);
        eq &= eq - 1;
        --take;
      }
      keep[w] |= add;
    }
    __syncthreads();
  }
  // movers: kept, slot >= budget - 1; free: not kept, slot < budget - 1, and slot budget - 1
  const int edge = a.budget - 1, we = edge / 32;
  const uint32_t below = (1u << (edge & 31)) - 1u;
  auto mover = [&](int w) { return w < we ? 0u : w == we ? keep[w] & ~below : keep[w]; };
  auto empty = [&](int w) { return w < we ? ~keep[w] : (~keep[w] & below) | (1u << (edge & 31)); };
  int* pref_f = reinterpret_cast<int*>(equal);
  if (warp == 0) {
    const int moves = warp_scan(nw, pref_m, [&](int w) { return __popc(mover(w)); });
    if (lane == 0) s_moves = moves;
  } else if (warp == 1) {
    warp_scan(we + 1, pref_f, [&](int w) { return __popc(empty(w)); });
  }
  __syncthreads();
  // Moves r = 0 .. moves - 1, the last one (slot n - 1 to slot budget - 1) together with the first.
  const int moves = s_moves, rounds = max(moves - 1, 1);
  const bool pair = moves > 1;
  auto place = [&](int r, int* src, int* dst, auto nth) {
    const int wm = find_word(pref_m, 0, nw, r), wf = find_word(pref_f, 0, we + 1, r);
    *src = wm * 32 + nth(mover(wm), r - pref_m[wm]);
    *dst = wf * 32 + nth(empty(wf), r - pref_f[wf]);
  };
  // The codes in pieces of up to 32 x 8 vectors, dealt out to the cluster's warps, a piece's loads in flight together:
  // of a block of more, a part; of smaller ones, as many moves as fit, but not so many that warps have none.  A lane
  // finds its move's slots for the others, and takes the move's scale and weight (with K) or number (with V).
  const int nv = a.block * a.hd / 16, per = (nv + 255) / 256;  // vectors of a block, and pieces
  const int warps = a.ctas * kEvictThreads / 32, me = warp * a.ctas + rank;
  const int group = !kGroups || 2 * rounds <= warps ? 1 : min(a.group, (2 * rounds + warps - 1) / warps);
  const int pieces = (group == 1 ? rounds : (rounds + group - 1) / group) * 2 * per;
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  for (int w = me; w < pieces; w += warps) {
    const int r0 = w / (2 * per) * group, q = w % (2 * per), m = min(group, rounds - r0);
    const int x = q >= per, first = (x ? q - per : q) * 256 + lane;
    int src = 0, dst = 0, left = m;  // moves of the piece
    if (!kGroups || m == 1) place(r0, &src, &dst, nth_bit_warp);
    else if (lane < m) place(r0 + lane, &src, &dst, nth_bit);
    uint4* rows = reinterpret_cast<uint4*>((x ? a.code[1] : a.code[0]) + unit * a.capacity * a.hd);
    uint32_t* scale = reinterpret_cast<uint32_t*>(x ? a.scale[1] : a.scale[0]) + unit * nblk;
    uint32_t* other = (x ? reinterpret_cast<uint32_t*>(a.ids) : reinterpret_cast<uint32_t*>(a.weight)) + unit * nblk;
    if (!kGroups && lane == 1) scale = other;  // two lanes for the one move
    const bool tails = x ? q == per : q == 0;
    bool again = r0 == 0 && pair;
    for (;;) {
      uint4 v[8];
      uint32_t t0 = 0u, t1 = 0u;
      if (tails && lane < (kGroups ? left : 2)) {
        t0 = scale[src];
        if (kGroups) t1 = other[src];
      }
      if (!kGroups || left == 1) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (first + 32 * k < nv) v[k] = rows[static_cast<int64_t>(src) * nv + first + 32 * k];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (first + 32 * k < nv) rows[static_cast<int64_t>(dst) * nv + first + 32 * k] = v[k];
      } else {  // blocks of 128 vectors at most: 32 bits number a unit's
        auto vector = [&](int k, int slot, int* j) {
          const int at = first + 32 * k;
          *j = at * a.magic >> 16;
          return __shfl_sync(0xffffffffu, slot, *j) * nv + at - *j * nv;
        };
        int j;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int from = vector(k, src, &j);
          if (j < left) v[k] = rows[from];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int to = vector(k, dst, &j);
          if (j < left) rows[to] = v[k];
        }
      }
      if (tails && lane < (kGroups ? left : 2)) {
        scale[dst] = t0;
        if (kGroups) other[dst] = t1;
      }
      // the last move goes with the first one, thread by thread
      if (!again) break;
      again = false;
      left = 1;
      src = n - 1;
      dst = edge;
    }
  }
  if (writes_len) a.lens_out[b] = static_cast<int32_t>(len - static_cast<int64_t>(n - a.budget) * a.block);
}

}  // namespace

// -------------------------------------------------------------- launchers
// Every kernel here waits (griddepcontrol.wait) before it reads or writes what an
// earlier one may have written or read (the joining kernel's lengths apart, see
// there), and lets the next one start its own preparation: launched
// programmatically, the calls of a decode step hide each other's launch and set-up
// (append of one token 2.6 -> 2.3 us, a short attention 10.4 -> 9.9; the latter is 8.9
// since its start was shortened).
template <typename... P, typename... A>
static xkv_status launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, int cluster,
                         const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? XKV_OK : XKV_ERR_CUDA;
}

// Warps and vectors a thread for the rows that one block can get: a warp up to
// 128 vectors of sixteen (16 rows of 128), 128 threads up to 512, 256 for more.
template <typename T>
static xkv_status append_typed(const AppendArgs& a, int64_t n_new, int block, int64_t blocks, cudaStream_t st) {
  const int vecs = static_cast<int>(std::min<int64_t>(n_new, block)) * a.hd / 16;
  const int64_t grid = vecs <= 128 ? (blocks + 3) / 4 : blocks;
  if (grid > 0x7FFFFFFF) return XKV_ERR_UNSUPPORTED;
  const unsigned g = static_cast<unsigned>(grid);
  return vecs <= 32     ? launch(kv8_append_kernel<T, 1, 1>, g, 128, 0, st, 1, a)
         : vecs <= 64   ? launch(kv8_append_kernel<T, 2, 1>, g, 128, 0, st, 1, a)
         : vecs <= 128  ? launch(kv8_append_kernel<T, 4, 1>, g, 128, 0, st, 1, a)
         : vecs <= 256  ? launch(kv8_append_kernel<T, 2, 4>, g, 128, 0, st, 1, a)
         : vecs <= 512  ? launch(kv8_append_kernel<T, 4, 4>, g, 128, 0, st, 1, a)
         : vecs <= 1024 ? launch(kv8_append_kernel<T, 4, 8>, g, 256, 0, st, 1, a)
                        : launch(kv8_append_kernel<T, 8, 8>, g, 256, 0, st, 1, a);
}

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
  a.B = p->batch;
  a.Hkv = p->n_kv_heads;
  a.hd = p->head_dim;
  a.block_log2 = 31 - __builtin_clz(static_cast<unsigned>(p->block));
  a.vpr_magic = static_cast<uint32_t>(((1 << 20) + p->head_dim / 16 - 1) / (p->head_dim / 16));
  const int64_t nb = (n_new + p->block - 2) / p->block + 1;
  a.nb = static_cast<int>(std::min(nb, p->capacity / p->block));
  a.status = device_status_ptr();
  const int64_t blocks = static_cast<int64_t>(p->batch) * p->n_kv_heads * 2 * a.nb;
  return dt == XKV_BF16 ? append_typed<__nv_bfloat16>(a, n_new, p->block, blocks, st)
                        : append_typed<float>(a, n_new, p->block, blocks, st);
}

KV8Plan kv8_plan(const xkv_kv8_params* p, int n_q_heads) {
  KV8Plan r{};
  const int gq = n_q_heads / p->n_kv_heads, hd = p->head_dim;
  const int64_t units = static_cast<int64_t>(p->batch) * p->n_kv_heads;
  r.tiles_cap = (p->capacity + kTile - 1) / kTile;
  r.ctas = std::min(num_sms(), kMaxSlots / 2);
  const int spt = kTile / sub_rows(p->block);
  const size_t slots = 2 * static_cast<size_t>(units + r.ctas);
  r.off_ml = align_up(slots * gq * hd * 4);
  r.off_wpart = r.off_ml + align_up(slots * gq * 8);
  r.off_wref = r.off_wpart + align_up(static_cast<size_t>(units) * r.tiles_cap * spt * gq * 4);
  r.off_span = r.off_wref + align_up(static_cast<size_t>(units) * r.tiles_cap * gq * 4);
  r.bytes = r.off_span + align_up(static_cast<size_t>(units) * 8);
  return r;
}

template <typename T, int GQ, int HDA>
static xkv_status attend_tc_shape(const AttendArgs& a, const CUtensorMap* maps, cudaStream_t st) {
  constexpr int smem = AttendShape<T, GQ, HDA>::smem;
  if (cudaFuncSetAttribute(kv8_attend_tc_kernel<T, GQ, HDA>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess)
    return XKV_ERR_CUDA;
  return launch(kv8_attend_tc_kernel<T, GQ, HDA>, a.ctas, kAttendThreads, smem, st, 1, maps[0], maps[1], a);
}

template <typename T>
static xkv_status attend_tc(const AttendArgs& a, const CUtensorMap* maps, cudaStream_t st) {
  if (a.hd <= 128)
    return a.gq <= 4   ? attend_tc_shape<T, 4, 1>(a, maps, st)
           : a.gq <= 8 ? attend_tc_shape<T, 8, 1>(a, maps, st)
                       : attend_tc_shape<T, 16, 1>(a, maps, st);
  return a.gq <= 4   ? attend_tc_shape<T, 4, 2>(a, maps, st)
         : a.gq <= 8 ? attend_tc_shape<T, 8, 2>(a, maps, st)
                     : attend_tc_shape<T, 16, 2>(a, maps, st);
}

xkv_status kv8_attend_launch(const xkv_kv8_params* p, const xkv_kv8_cache* c, const int32_t* lens, int n_q_heads,
                             xkv_dtype dt, const void* q, float* out, int accumulate, const KV8Plan& plan, void* ws,
                             cudaStream_t st) {
  AttendArgs a{};
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.q = q;
  a.lens = lens;
  char* w = static_cast<char*>(ws);
  a.part = reinterpret_cast<float*>(w);
  a.ml = reinterpret_cast<float2*>(w + plan.off_ml);
  if (accumulate) {
    a.wpart = reinterpret_cast<float*>(w + plan.off_wpart);
    a.wref = reinterpret_cast<float*>(w + plan.off_wref);
    a.weight = c->weight;
  }
  a.span = reinterpret_cast<int2*>(w + plan.off_span);
  a.out = out;
  a.capacity = p->capacity;
  a.B = p->batch;
  a.Hkv = p->n_kv_heads;
  a.gq = n_q_heads / p->n_kv_heads;
  a.hd = p->head_dim;
  a.block = p->block;
  a.tiles_cap = static_cast<int>(plan.tiles_cap);
  a.ctas = plan.ctas;
  a.q_scale = kLog2e / std::sqrt(static_cast<float>(p->head_dim));
  a.status = device_status_ptr();
  CUtensorMap maps[2];
  for (int x = 0; x < 2; ++x) {
    const uint64_t dims[3] = {static_cast<uint64_t>(p->head_dim), static_cast<uint64_t>(p->capacity),
                              static_cast<uint64_t>(p->batch) * p->n_kv_heads};
    const uint64_t str[2] = {static_cast<uint64_t>(p->head_dim), static_cast<uint64_t>(p->head_dim) * p->capacity};
    const uint32_t box[3] = {128, kTile, 1};
    if (!make_tmap(&maps[x], CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, x ? c->v : c->k, dims, str, box,
                   CU_TENSOR_MAP_SWIZZLE_128B))
      return XKV_ERR_CUDA;
  }
  const xkv_status s = dt == XKV_BF16 ? attend_tc<__nv_bfloat16>(a, maps, st) : attend_tc<float>(a, maps, st);
  if (s != XKV_OK) return s;
  // joining: heads to a CTA so that its grid is about what the card holds at once (four CTAs an SM)
  const int64_t units = static_cast<int64_t>(p->batch) * p->n_kv_heads;
  int heads = 1;
  while (heads < 8 && heads < a.gq && units * ((a.gq + heads - 1) / heads) > 4 * num_sms()) heads *= 2;
  const int head_ctas = (a.gq + heads - 1) / heads;
  int wy = 0;
  if (accumulate) {
    const int64_t nblk = p->capacity / p->block;
    wy = static_cast<int>(std::min<int64_t>((nblk + kWeightBlocks - 1) / kWeightBlocks, 64));
  }
  return launch(kv8_combine_kernel, dim3(static_cast<unsigned>(units), head_ctas + wy), kCombineThreads, 0, st, 1, a,
                heads, head_ctas);
}

xkv_status kv8_evict_launch(const xkv_kv8_params* p, const xkv_kv8_cache* c, const int32_t* lens, int budget, int sink,
                            int recent, int32_t* lens_out, cudaStream_t st) {
  const int64_t nblk = p->capacity / p->block;
  if (nblk > kEvictMaxBlocks || static_cast<int64_t>(p->batch) * p->n_kv_heads * kEvictCtas > 0x7FFFFFFF)
    return XKV_ERR_UNSUPPORTED;
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
  a.keys = nblk > kEvictHeld * kEvictThreads ? static_cast<int>(std::min(nblk, kEvictKeys)) : 0;
  const size_t smem = static_cast<size_t>((nblk + 31) / 32) * 3 * 4 + static_cast<size_t>(a.keys) * 4;
  const int nv = p->block * p->head_dim / 16;
  a.group = nv > 128 ? 1 : std::min(256 / nv, 32);
  a.magic = (65535u + nv) / nv;
  // CTAs to a unit: up to eight, as long as each warp can get two pieces of the most blocks that can move, or, where
  // SMs are idle, two moves.  A CTA of its own costs each the selection: with eight for every unit, 144 units of 9
  // blocks took 17 us, with one 6 us; 60 units of 300 blocks (hd 48, 8 tokens each) cut to 150 take 16 us with eight
  // and 11 with two, 2 units of 128 blocks 7.6 with one and 7.1 with four.  Small blocks, whose selection is most of the
  // work, in one round of three CTAs an SM: 60 units of 5113 such blocks cut to 4758 30 us with four, 42 with eight.
  // (With large blocks and ragged lengths the CTAs of sequences within the budget leave at once: 26 us with eight for
  // 64 units, 40 with fewer.)
  const int64_t moves = std::min<int64_t>(budget, std::max<int64_t>(nblk - budget + 1, 1));
  const int64_t parts = 2 * moves * ((nv + 255) / 256), units = static_cast<int64_t>(p->batch) * p->n_kv_heads;
  a.ctas = 1;
  while (a.ctas < kEvictCtas && (a.group == 1 || 2 * a.ctas * units <= 3 * num_sms()) && parts > 2 * a.ctas * (kEvictThreads / 32) *
                                            (2 * a.ctas * units <= num_sms() ? 1 : a.group))
    a.ctas *= 2;
  auto* kernel = a.group > 1 ? kv8_evict_kernel<true> : kv8_evict_kernel<false>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kEvictMaxBlocks / 32 * 3 * 4 + kEvictKeys * 4)) != cudaSuccess)
    return XKV_ERR_CUDA;
  return launch(kernel, dim3(static_cast<unsigned>(units) * a.ctas), kEvictThreads, smem, st, a.ctas, a);
}

}  // namespace xkv
