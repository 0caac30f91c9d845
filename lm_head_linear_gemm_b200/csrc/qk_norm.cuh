// Queries and keys normed per head and rotated by position in one pass, and the backward of both.
//
// Both kernels are bound by HBM: a row is read once (16 elements for each lane: eight pairs of the
// rotation), reduced over the LANES lanes that hold it, and written once.  A warp takes the heads of
// one token, 32 / LANES rows at a pass, so that the token's cosines and sines are formed once per
// warp and stay in registers across its heads.  The rows come through a ring in shared memory that
// each lane fills for itself some passes ahead, across heads and tokens, so that what is in flight
// takes no registers; the arithmetic is in pairs of fp32 (two operations in an instruction): one at
// a time it took longer than the memory.
//
// 16 x 1024 tokens of 32 + 8 heads of 128 in bf16, one B200 (a copy runs at 6.57 TB/s), a call: forward
// 59 us, 5.7 TB/s; backward 90 to 96 us, 5.2 to 5.6 TB/s, with half of the issue slots taken.  In fp32
// 116 us, 5.8 TB/s, and 172, 5.9.  One token: 3.8 us of GPU time, the latency of a launch, a row and a
// store.  The backward is held to 128 registers (two blocks on an SM) and all but two of its 40
// instances spill a little: 8 to 28 bytes a thread, 40 to 76 with 3, 5, 6 or 10 lanes to a row.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "packed.cuh"

namespace flce {


constexpr int kQkWarps = 8;            // warps of a block
constexpr int kQkBlocks = 2;           // of an SM
constexpr int kQkMaxParts = 592;       // dgamma partials of one launch (4 blocks on each of 148 SMs)

struct QkView {
  void* ptr;
  long long batch, token, head;
};

// Division of n < 2^31 by a divisor known at the launch: with 2^(shift - 31) the power of two not
// below d and mul = ceil(2^shift / d), n mul / 2^shift has the quotient (mul d - 2^shift is below
// 2^(shift - 31), so n times it stays below 2^shift).
struct QkDivisor {
  uint32_t d, mul, shift;
  __device__ __forceinline__ uint32_t quotient(uint32_t n) const {
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * mul) >> shift);
  }
};

struct QkArgs {
  QkView q, k, dq, dk, yq, yk;         // inputs; gradients of the outputs (backward); results
  const void* gamma_q;
  const void* gamma_k;
  const float* inv_freq;
  const long long* positions;
  long long positions_batch;
  QkDivisor T, segs;                   // tokens of a sequence; segments of a token's passes
  uint32_t items;                      // tokens of all sequences x segments of a token's passes
  uint32_t seg_passes;
  int Hq, Hk, D, rot;
  float eps;
  int gamma_f32;
  float* partial;                      // [grid][2][D] (backward)
};

// 16 elements of a row as loaded, in chunks of 16 bytes: two of bf16, four of fp32.
template <typename T>
struct QkRaw {
  static constexpr int kChunks = sizeof(T), kChunk = 16 / sizeof(T);
  uint4 c[kChunks];
};
// The same as eight pairs of the rotation, two pairs to an element: pair 2i is (a[i].x, b[i].x),
// pair 2i + 1 (a[i].y, b[i].y).
struct QkPairs {
  float2 a[4], b[4];
};

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <bool INTER>
__device__ __forceinline__ void qk_unpack(const QkRaw<__nv_bfloat16>& r, QkPairs& p) {
  const uint32_t w[8] = {r.c[0].x, r.c[0].y, r.c[0].z, r.c[0].w,
                         r.c[1].x, r.c[1].y, r.c[1].z, r.c[1].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (INTER) {                       // a word is a pair
      p.a[i] = make_float2(bf16_low(w[2 * i]), bf16_low(w[2 * i + 1]));
      p.b[i] = make_float2(bf16_high(w[2 * i]), bf16_high(w[2 * i + 1]));
    } else {                           // a word of each half is two pairs
      p.a[i] = make_float2(bf16_low(w[i]), bf16_high(w[i]));
      p.b[i] = make_float2(bf16_low(w[4 + i]), bf16_high(w[4 + i]));
    }
  }
}
template <bool INTER>
__device__ __forceinline__ void qk_unpack(const QkRaw<float>& r, QkPairs& p) {
  float f[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[4 * i] = __uint_as_float(r.c[i].x);
    f[4 * i + 1] = __uint_as_float(r.c[i].y);
    f[4 * i + 2] = __uint_as_float(r.c[i].z);
    f[4 * i + 3] = __uint_as_float(r.c[i].w);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (INTER) {
      p.a[i] = make_float2(f[4 * i], f[4 * i + 2]);
      p.b[i] = make_float2(f[4 * i + 1], f[4 * i + 3]);
    } else {
      p.a[i] = make_float2(f[2 * i], f[2 * i + 1]);
      p.b[i] = make_float2(f[8 + 2 * i], f[8 + 2 * i + 1]);
    }
  }
}
__device__ __forceinline__ uint32_t bf16_word(float low, float high) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(low, high);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool INTER>
__device__ __forceinline__ void qk_pack(const QkPairs& p, QkRaw<__nv_bfloat16>& r) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (INTER) {
      w[2 * i] = bf16_word(p.a[i].x, p.b[i].x);
      w[2 * i + 1] = bf16_word(p.a[i].y, p.b[i].y);
    } else {
      w[i] = bf16_word(p.a[i].x, p.a[i].y);
      w[4 + i] = bf16_word(p.b[i].x, p.b[i].y);
    }
  }
  r.c[0] = make_uint4(w[0], w[1], w[2], w[3]);
  r.c[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
template <bool INTER>
__device__ __forceinline__ void qk_pack(const QkPairs& p, QkRaw<float>& r) {
  float f[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[INTER ? 4 * i : 2 * i] = p.a[i].x;
    f[INTER ? 4 * i + 2 : 2 * i + 1] = p.a[i].y;
    f[INTER ? 4 * i + 1 : 8 + 2 * i] = p.b[i].x;
    f[INTER ? 4 * i + 3 : 8 + 2 * i + 1] = p.b[i].y;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.c[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                        __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
}

// Where the 16 elements of unit u of a row lie: in chunks of 16 bytes, the same chunk of the row's
// units side by side, so that a load of one chunk by all lanes covers whole sectors.  The first
// rot/16 units hold the rotated elements; the first half of a unit's chunks lies in the first half of
// these elements and the other chunks at the same places of the second, where halves are paired
// with one another.
template <typename T, bool INTER>
struct QkUnit {
  static constexpr int kChunks = QkRaw<T>::kChunks, kChunk = QkRaw<T>::kChunk;
  bool turned;
  int base, step;                      // chunk i at base + i step
  __device__ QkUnit(int u, int D, int rot) {
    const int units = rot / 16;
    turned = u < units;
    base = turned ? kChunk * u : rot + kChunk * (u - units);
    step = kChunk * (turned ? units : D / 16 - units);
  }
  __device__ __forceinline__ int chunk(int i) const { return base + i * step; }
  // The place of element j of QkPairs' a (j < 8) or b (j - 8).
  __device__ __forceinline__ int element(int j) const {
    const int i = INTER ? 2 * (j & 7) + (j >> 3) : j;      // among the 16 as loaded
    return chunk(i / kChunk) + i % kChunk;
  }
  // The first of the pairs 2k, 2k + 1 of a turned unit, which are neighbours.
  __device__ __forceinline__ int pair(int k) const {
    const int i = INTER ? 4 * k : 2 * k;
    const int at = base + i / kChunk * step + i % kChunk;
    return INTER ? at / 2 : at;
  }
};

template <typename T, int LANES, bool INTER>
struct QkLane : QkUnit<T, INTER> {
  int group;
  bool active;
  __device__ QkLane(int lane, int D, int rot)
      : QkUnit<T, INTER>(lane % LANES < D / 16 ? lane % LANES : 0, D, rot),
        group(lane / LANES),
        active(lane % LANES < D / 16 && lane < 32 / LANES * LANES) {}
};

template <typename T, bool INTER>
__device__ __forceinline__ void qk_store(T* chunk, int step, const QkPairs& p) {
  QkRaw<T> r;
  qk_pack<INTER>(p, r);
#pragma unroll
  for (int i = 0; i < QkRaw<T>::kChunks; ++i)
    *reinterpret_cast<uint4*>(chunk + i * step) = r.c[i];
}

// cos and sin of every pair at this position, formed once by the warp.  The angle in turns is a
// product in 64 bits (with the frequencies in turns, s_freq) less its nearest integer, so that far
// positions lose nothing.  Of what is left, |x| <= 1/2 turn, the sine and cosine are taken in fp32;
// what fp32 loses of x (up to 2^-26 turns, 9e-8 rad, more than a sine's own rounding) turns them on:
// its square is below 2^-46.
__device__ __forceinline__ void qk_angles(int lane, double pos, const double* s_freq, int half,
                                          float2* s_cs) {
  __syncwarp();                        // the previous token's values are read
  for (int i = lane; i < half; i += 32) {
    const double turns = pos * s_freq[i];
    const double rest = turns - rint(turns);
    const float part = static_cast<float>(rest);
    const float low = static_cast<float>(rest - static_cast<double>(part)) * 6.283185307f;
    float c, s;
    sincospif(2.f * part, &s, &c);
    s_cs[i] = make_float2(fmaf(-s, low, c), fmaf(c, low, s));
  }
  __syncwarp();
}
// Those of the lane's eight pairs (1 and 0 behind the rotated part).
template <typename T, bool INTER>
__device__ __forceinline__ void qk_cos_sin(const QkUnit<T, INTER>& at, const float2* s_cs,
                                           float2 (&c)[4], float2 (&s)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    c[k] = make_float2(1.f, 1.f), s[k] = make_float2(0.f, 0.f);
    if (at.turned) {
      const float4 w = *reinterpret_cast<const float4*>(s_cs + at.pair(k));
      c[k] = make_float2(w.x, w.z);
      s[k] = make_float2(w.y, w.w);
    }
  }
}
// gamma's 16 elements of this lane, from fp32 in shared memory in the rows' order.
template <typename T, bool INTER>
__device__ __forceinline__ void qk_gamma(const float* s_gamma, const QkUnit<T, INTER>& at,
                                         QkPairs& g) {
  QkRaw<float> r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.c[i] = *reinterpret_cast<const uint4*>(
        s_gamma + at.chunk(4 * i / QkRaw<T>::kChunk) + 4 * i % QkRaw<T>::kChunk);
  qk_unpack<INTER>(r, g);
}

// The sum over a row's lanes, in all of them.  Where they are no power of two, the first takes from
// behind while there is any, and hands it round.
template <int LANES>
__device__ __forceinline__ float qk_sum(float v) {
  if ((LANES & (LANES - 1)) == 0) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  const int lane = threadIdx.x & 31, u = lane % LANES;
#pragma unroll
  for (int o = LANES > 8 ? 8 : LANES > 4 ? 4 : 2; o > 0; o >>= 1) {
    const float behind = __shfl_down_sync(0xffffffffu, v, o);
    if (u + o < LANES) v += behind;
  }
  return __shfl_sync(0xffffffffu, v, lane - u);
}

// ------------------------------------------------------------------------------ the ring
template <typename T, bool BWD>
struct QkRing {
  static constexpr int kRow = 16 * sizeof(T);              // bytes of a lane's 16 elements
  static constexpr int kSlot = 32 * kRow * (BWD ? 2 : 1);  // x, and dy
  // Three passes: more in flight ran slower (forward of 16k tokens 59 us with 3, 62 with 2, 64 with
  // 4, 65 with 8 slots).  fp32 backward: two, so that two blocks fit an SM up to heads of 256 (above,
  // with 22 KB for angles and gammas, one does).
  static constexpr int kSlots = BWD && sizeof(T) == 4 ? 2 : 3;
  static constexpr int kWarp = kSlots * kSlot;
  // the backward's sums of d xh: 16 elements of each lane for q and for k
  static constexpr int kSums = BWD ? 2 * 32 * 64 : 0;
  static constexpr int kBytes = kQkWarps * (kWarp + kSums);
};
// 16 bytes into shared memory: `bytes` (16 or 0) of them copied, the rest zeros.
__device__ __forceinline__ void qk_copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
// A lane's 16 elements into a slot (zeros where it has none) and from it, chunk by chunk of the warp:
// no two lanes of an access share a bank.
template <typename T>
__device__ __forceinline__ void qk_fetch(uint32_t slot, const T* chunk, int step, int bytes) {
#pragma unroll
  for (int i = 0; i < QkRaw<T>::kChunks; ++i) qk_copy16(slot + 512 * i, chunk + i * step, bytes);
}
template <typename T>
__device__ __forceinline__ void qk_take(const uint8_t* slot, QkRaw<T>& r) {
#pragma unroll
  for (int i = 0; i < QkRaw<T>::kChunks; ++i)
    r.c[i] = *reinterpret_cast<const uint4*>(slot + 512 * i);
}

// An item: the passes [first, end) of one token's, those of the queries before those of the keys.
struct QkItem {
  uint32_t b, t;
  int first, end;
  template <int ROWS>
  __device__ __forceinline__ void find(const QkArgs& p, uint32_t item) {
    const uint32_t token = p.segs.quotient(item);
    const uint32_t seg = item - token * p.segs.d;
    b = p.T.quotient(token);
    t = token - b * p.T.d;
    first = static_cast<int>(seg * p.seg_passes);
    end = min(first + static_cast<int>(p.seg_passes),
              (p.Hq + ROWS - 1) / ROWS + (p.Hk + ROWS - 1) / ROWS);
  }
  // This kind's passes (0 queries, 1 keys): from, and how many.
  __device__ __forceinline__ int part(int kind, int q_passes, int* from) const {
    const int lo = kind ? max(first - q_passes, 0) : first;
    *from = lo;
    return (kind ? end - q_passes : min(end, q_passes)) - lo;
  }
  __device__ __forceinline__ long long at(const QkView& v) const {
    return static_cast<long long>(b) * v.batch + static_cast<long long>(t) * v.token;
  }
};
__device__ __forceinline__ double qk_position(const QkArgs& p, const QkItem& it) {
  return p.positions != nullptr
             ? static_cast<double>(p.positions[it.b * p.positions_batch + it.t])
             : static_cast<double>(it.t);
}

// Brings a warp's rows, pass by pass through its items, into the ring.
template <typename T, int LANES, bool INTER, bool BWD>
struct QkFeed {
  static constexpr int ROWS = 32 / LANES;
  using Ring = QkRing<T, BWD>;
  uint32_t item;                       // the next item
  uint32_t slot, begin;                // this lane's place in the next slot, and in the first
  QkItem it;
  int kind, left, rows;                // of the present item: its kind, passes left, and how many
                                       // rows from this lane's on there are in it
  const T *x, *d;
  long long x_step, d_step;            // of a pass
  // Nothing more to bring: passes without rows.  They copy no byte, but their addresses have to be
  // aligned all the same, which a lone head's stride need not be: they stay at an array's start.
  __device__ __forceinline__ void rest(const QkArgs& p) {
    x = static_cast<const T*>(p.Hq > 0 ? p.q.ptr : p.k.ptr);
    d = static_cast<const T*>(p.Hq > 0 ? p.dq.ptr : p.dk.ptr);
    x_step = d_step = 0;
    left = 0x7fffffff;
    rows = 0;
  }
  // The next kind, or the next item's first.
  __device__ __forceinline__ void refill(const QkArgs& p, const QkLane<T, LANES, INTER>& ln,
                                         int q_passes, uint32_t stride) {
    do {
      if (kind == 1) {
        if (item >= p.items) return rest(p);
        it.find<ROWS>(p, item);
        item += stride;
        kind = -1;
      }
      ++kind;
      int from;
      left = it.part(kind, q_passes, &from);
      // a lane without rows stays at the first head: a lone head's stride need not be aligned
      int row = from * ROWS + ln.group;
      rows = ln.active ? (kind ? p.Hk : p.Hq) - row : 0;
      if (rows <= 0) row = 0;
      const QkView& v = kind ? p.k : p.q;
      x = static_cast<const T*>(v.ptr) + (it.at(v) + row * v.head + ln.base);
      x_step = ROWS * v.head;
      if (BWD) {
        const QkView& g = kind ? p.dk : p.dq;
        d = static_cast<const T*>(g.ptr) + (it.at(g) + row * g.head + ln.base);
        d_step = ROWS * g.head;
      }
    } while (left <= 0);
  }
  __device__ __forceinline__ void one(const QkArgs& p, const QkLane<T, LANES, INTER>& ln,
                                      int q_passes, uint32_t stride) {
    if (left <= 0) refill(p, ln, q_passes, stride);
    const int bytes = rows > 0 ? 16 : 0;
    qk_fetch<T>(slot, x, ln.step, bytes);
    x += x_step;
    if (BWD) {
      qk_fetch<T>(slot + 32 * Ring::kRow, d, ln.step, bytes);
      d += d_step;
    }
    --left;
    rows -= ROWS;
    slot = slot == begin + (Ring::kSlots - 1) * Ring::kSlot ? begin : slot + Ring::kSlot;
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
};

// The sums over the block's rows of one gamma's gradient: over the warps in order, and in each over
// the lanes that held the element, in order.  Always the same order.
template <typename T, int LANES, bool INTER>
__device__ __forceinline__ void qk_block_dgamma(const QkArgs& p, const float* s_sums, int kind,
                                                float* out) {
  for (int e = threadIdx.x; e < p.D; e += 32 * kQkWarps) {
    const int u = e % (p.D / 16), j = e / (p.D / 16);      // element j of unit u
    float sum = 0.f;
    for (int w = 0; w < kQkWarps; ++w)
      for (int g = 0; g < 32 / LANES; ++g)
        sum += s_sums[(((w * 2 + kind) * 4 + j / 4) * 32 + g * LANES + u) * 4 + j % 4];
    out[QkUnit<T, INTER>(u, p.D, p.rot).element(j)] = sum;
  }
}

// Forward: y = rotate(x rstd gamma), with gamma in the coefficients: y_a = rstd (x_a ca + x_b sb),
// y_b = rstd (x_a sa + x_b cb).  Backward: with d the output's gradient rotated back, g = d gamma
// and xh = x rstd: dx = rstd (g - xh mean(g xh)), and the sums of d xh for dgamma.
template <typename T, int LANES, bool INTER, bool BWD>
__global__ void __launch_bounds__(32 * kQkWarps, kQkBlocks)
    qk_norm_rope_kernel(const QkArgs p) {
  using Ring = QkRing<T, BWD>;
  constexpr int ROWS = 32 / LANES;
  extern __shared__ __align__(16) uint8_t s_ring[];
  __shared__ __align__(16) float2 s_cs[kQkWarps][8 * LANES];
  __shared__ __align__(16) float s_gamma[2][16 * LANES];
  __shared__ double s_freq[8 * LANES];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const QkLane<T, LANES, INTER> ln(lane, p.D, p.rot);
  const float inv_d = 1.f / static_cast<float>(p.D);
  const int q_passes = (p.Hq + ROWS - 1) / ROWS;
  const uint32_t stride = gridDim.x * kQkWarps;
  uint8_t* ring = s_ring + warp * Ring::kWarp;
  float4* sums = reinterpret_cast<float4*>(s_ring + kQkWarps * Ring::kWarp) + warp * 2 * 4 * 32 + lane;
  uint32_t item = blockIdx.x * kQkWarps + warp;

  // the sum over the blocks may be made ready to start (it waits for this launch's end)
  if (BWD) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  QkFeed<T, LANES, INTER, BWD> feed;
  feed.item = item;
  feed.slot = feed.begin = static_cast<uint32_t>(__cvta_generic_to_shared(ring + 16 * lane));
  feed.kind = 1;
  feed.left = 0;
#pragma unroll 1
  for (int i = 0; i < Ring::kSlots - 1; ++i) feed.one(p, ln, q_passes, stride);
  if (BWD)
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[32 * i] = make_float4(0.f, 0.f, 0.f, 0.f);

  QkItem it;
  double pos = 0.0;
  if (item < p.items) {
    it.find<ROWS>(p, item);
    pos = qk_position(p, it);
  }
  for (int i = threadIdx.x; i < p.rot / 2; i += 32 * kQkWarps)
    s_freq[i] = static_cast<double>(p.inv_freq[i]) * 0.15915494309189533577;   // 1 / (2 pi)
  for (int e = threadIdx.x; e < 2 * p.D; e += 32 * kQkWarps) {
    const int kind = e >= p.D, at = e - kind * p.D;
    const void* gamma = kind ? p.gamma_k : p.gamma_q;
    s_gamma[kind][at] =
        gamma == nullptr ? 1.f
        : p.gamma_f32    ? static_cast<const float*>(gamma)[at]
                         : __bfloat162float(static_cast<const __nv_bfloat16*>(gamma)[at]);
  }
  __syncthreads();

  const uint8_t* slot = ring + 16 * lane;
#pragma unroll 1
  for (; item < p.items; item += stride) {
    it.find<ROWS>(p, item);
    qk_angles(lane, pos, s_freq, p.rot / 2, s_cs[warp]);
    if (stride < p.items - item) {     // the next item's position, long before it is needed
      QkItem then;
      then.find<ROWS>(p, item + stride);
      pos = qk_position(p, then);
    }
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
      int from;
      const int passes = it.part(kind, q_passes, &from);
      if (passes <= 0) continue;
      const QkView& v = kind ? p.yk : p.yq;
      const int row = from * ROWS + ln.group;
      int rows = ln.active ? (kind ? p.Hk : p.Hq) - row : 0;
      T* y = static_cast<T*>(v.ptr) + (it.at(v) + row * v.head + ln.base);
      const long long step = ROWS * v.head;
      // forward: the coefficients of x_a and x_b in y_a and y_b; backward: cos and sin
      float2 ca[4], sa[4], cb[4], sb[4];
      qk_cos_sin<T, INTER>(ln, s_cs[warp], ca, sa);
      if (!BWD) {
        QkPairs g;
        qk_gamma<T, INTER>(s_gamma[kind], ln, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cb[i] = mul2(g.b[i], ca[i]);
          sb[i] = mul2(g.b[i], make_float2(-sa[i].x, -sa[i].y));
          ca[i] = mul2(g.a[i], ca[i]);
          sa[i] = mul2(g.a[i], sa[i]);
        }
      }
      QkPairs acc;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc.a[i] = acc.b[i] = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int pass = 0; pass < passes; ++pass) {
        feed.one(p, ln, q_passes, stride);
        asm volatile("cp.async.wait_group %0;" ::"n"(Ring::kSlots - 1) : "memory");
        const uint8_t* from = slot;
        slot = slot == ring + (Ring::kSlots - 1) * Ring::kSlot + 16 * lane
                   ? ring + 16 * lane
                   : slot + Ring::kSlot;
        const bool on = rows > 0;
        QkRaw<T> raw;
        QkPairs f;
        qk_take(from, raw);
        qk_unpack<INTER>(raw, f);
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fma2(f.b[i], f.b[i], fma2(f.a[i], f.a[i], ss));
        if (!BWD) {
          const float2 rstd = both(rsqrtf(fmaf(qk_sum<LANES>(ss.x + ss.y), inv_d, p.eps)));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 a = mul2(f.a[i], rstd), b = mul2(f.b[i], rstd);
            f.a[i] = fma2(a, ca[i], mul2(b, sb[i]));
            f.b[i] = fma2(a, sa[i], mul2(b, cb[i]));
          }
        } else {
          QkPairs d, gd;
          qk_take(from + 32 * Ring::kRow, raw);
          qk_unpack<INTER>(raw, d);
          float2 dot = make_float2(0.f, 0.f);
          qk_gamma<T, INTER>(s_gamma[kind], ln, gd);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 a = d.a[i], minus = make_float2(-a.x, -a.y);
            d.a[i] = fma2(a, ca[i], mul2(d.b[i], sa[i]));
            d.b[i] = fma2(minus, sa[i], mul2(d.b[i], ca[i]));
            gd.a[i] = mul2(d.a[i], gd.a[i]);
            gd.b[i] = mul2(d.b[i], gd.b[i]);
            dot = fma2(gd.b[i], f.b[i], fma2(gd.a[i], f.a[i], dot));
          }
          const float sum = qk_sum<LANES>(ss.x + ss.y), sdot = qk_sum<LANES>(dot.x + dot.y);
          const float rstd = rsqrtf(fmaf(sum, inv_d, p.eps));
          const float mean = sdot * rstd * inv_d;          // mean_j(g xh)
          // a row beyond the heads adds nothing: its rstd may be infinite
          const float2 r = both(on ? rstd : 0.f), m = both(-mean);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 xa = mul2(f.a[i], r), xb = mul2(f.b[i], r);
            acc.a[i] = fma2(d.a[i], xa, acc.a[i]);
            acc.b[i] = fma2(d.b[i], xb, acc.b[i]);
            f.a[i] = mul2(r, fma2(xa, m, gd.a[i]));
            f.b[i] = mul2(r, fma2(xb, m, gd.b[i]));
          }
        }
        if (on) qk_store<T, INTER>(y, ln.step, f);
        rows -= ROWS;
        y += step;
      }
      if (BWD) {
        float4* to = sums + kind * 4 * 32;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 lo = i < 2 ? acc.a[2 * i] : acc.b[2 * i - 4];
          const float2 hi = i < 2 ? acc.a[2 * i + 1] : acc.b[2 * i - 3];
          float4 w = to[32 * i];
          w.x += lo.x, w.y += lo.y, w.z += hi.x, w.w += hi.y;
          to[32 * i] = w;
        }
      }
    }
  }
  if (BWD) {
    __syncthreads();
    const float* all = reinterpret_cast<const float*>(s_ring + kQkWarps * Ring::kWarp);
    float* out = p.partial + static_cast<size_t>(blockIdx.x) * 2 * p.D;
    qk_block_dgamma<T, LANES, INTER>(p, all, 0, out);
    qk_block_dgamma<T, LANES, INTER>(p, all, 1, out + p.D);
  }
}

// dgamma (+)= the blocks' partials, 32 columns to a block of 32 x 32 threads: thread row y sums the
// parts y, y + 32, ... in order, then a warp sums a column's 32 by a fixed tree.  The launch before
// still writes the partials while this one starts, so they are no read-only data of this kernel:
// no __restrict__, and loads from L2 (__ldcg) behind the wait.
__global__ void __launch_bounds__(1024) qk_dgamma_kernel(const float* partial, int parts, int D,
                                                         float* dgamma_q, float* dgamma_k,
                                                         int accumulate) {
  __shared__ float s_sum[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");       // the partials are complete
  const int e = blockIdx.x * 32 + threadIdx.x;             // of 2 D columns: q's, then k's
  float acc = 0.f;
  if (e < 2 * D) {
#pragma unroll 4
    for (int b = threadIdx.y; b < parts; b += 32)
      acc += __ldcg(partial + static_cast<size_t>(b) * 2 * D + e);
  }
  s_sum[threadIdx.y][threadIdx.x] = acc;
  __syncthreads();
  const int at = blockIdx.x * 32 + threadIdx.y;            // this warp's column
  const float sum = qk_sum<32>(s_sum[threadIdx.x][threadIdx.y]);
  if (threadIdx.x != 0 || at >= 2 * D) return;
  float* out = at < D ? dgamma_q : dgamma_k;
  if (out == nullptr) return;
  const int i = at < D ? at : at - D;
  out[i] = accumulate ? out[i] + sum : sum;
}

}  // namespace flce
