// The AdamW step over many tensors in one launch, and the global gradient norm.
//
// Both are bound by HBM: every state, weight and gradient is read once and written once.  The
// tensors' descriptors travel in the launch's parameters, so a step needs no table on the device
// and may be captured with the pointers it was given.
//
// One B200 (a copy runs at 6.57 TB/s), a call: AdamW on 77 M bf16 weights, fp32 states and gradient
// 292 us, 6.3 TB/s; 8-bit states throughout, bf16 gradient 132 to 144 us with the clock, 5.4 to
// 5.9 TB/s, where the instructions (56% of the issue slots: conversions, roundings) and the memory
// bound it together; 236 M weights with master copies 629 to 638 us, 6.0 TB/s.  Norm of 236 M bf16
// values 74 to 76 us, 6.2 to 6.4 TB/s.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "packed.cuh"
#include "sm100.cuh"

namespace flce {

constexpr int kAdamTensors = 384;      // tensors of one launch: 28 KB of the 32 KB of parameters
constexpr int kFewTensors = 48;        // a launch of no more passes 4 KB instead (3 us less on the host)
constexpr int kAdamGroups = 16;
constexpr int kAdamThreads = 256;
constexpr int kAdamPart = 8 * kAdamThreads;    // elements of one step of a block's threads
constexpr int kAdamBlocks = 2;                 // of an SM
constexpr int kAdamRing = 73728;               // bytes of a block's ring
constexpr uint64_t kAdamWaitNs = 2000000000ull;   // bound of every wait in the kernel
constexpr int kAdamStages = 16;                // of the ring at most
constexpr int kStateBlock = 256;       // elements that share a scale: 8 for each lane of a warp
constexpr int kNormTensors = 1024;
constexpr int kNormThreads = 256;
constexpr int kNormChunk = 16384;
constexpr int kNormBlocks = 592;       // partial sums of one launch

struct AdamTensor {
  void* param;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* r_scale;
  float* master;
  long long n;
  uint8_t param_bf16, grad_bf16, state8, wide;
  uint8_t group, pad[3];
};
struct AdamGroup {
  const float* lr_device;
  double log_beta1, log_beta2;         // -inf for 0
  float lr, beta1, beta2, c1, c2, eps, weight_decay;   // c = 1 - beta
  float one;
};
// N: the tensors that a launch has room for.  PARTS: steps of the block's threads in a tile.  Tiles of
// two for long launches; of one, handed out one at a time, where a block has few: they start sooner
// and spread further (fp32, tiles of two and of one: 256 K elements 7.7 and 4.8 us, 2 M 15.1 and 12.6,
// 4 M 24.8 and 21.6; 8-bit states of 256 K 5.4 and 3.9, 4 M 12.6 and 12.2, but 8 M 19.7 and 21.0).
template <int N, int PARTS>
struct AdamArgs {
  static constexpr int kParts = PARTS;
  static constexpr int kTile = PARTS * kAdamPart;          // pass through the ring together
  static constexpr int kChunk = PARTS == 1 ? kTile : 2 * kTile;   // a block takes at a time
  static constexpr int kScales = 2 * kTile / kStateBlock;
  // the widest stage: four fp32 arrays, or fewer bytes and the scales
  static constexpr int kMaxStage = 16 * kTile + 256;
  static_assert(kMaxStage <= kAdamRing, "a stage of every kind fits the ring");
  static_assert(4 * kScales + 127 <= 256, "kMaxStage covers the scales");
  static_assert(kScales <= 32, "one lane each");
  uint32_t first[N];                   // the first of each tensor's chunks, which count through
  AdamTensor t[N];
  AdamGroup g[kAdamGroups];
  int count, groups;
  uint32_t chunks;
  // a stage of the ring: w, gradient, m, v or r codes, scales; sized for the launch's widest tensor
  uint32_t at_g, at_m, at_v, at_scales, stage, stages;
  int last;                            // the step's last launch counts it
  int skip_nonfinite;
  const float* grad_scale;
  long long* step;
  uint32_t* ticket;                    // scratch[0]; scratch[1] takes the status bits
};
static_assert(sizeof(AdamArgs<kAdamTensors, 2>) <= 32764, "a launch's parameters");
// What a group's elements need:
//   g = gs grad,  m = b1 m + c1 g,  v = b2 v + c2 g^2,  w = decay w + m / (da sqrt(v) + db)
// with da = 1 / (size sqrt(1 - beta2^t)), db = eps / size, size = -lr / (1 - beta1^t).
struct AdamScalars {
  float gs, b1, c1, b2, c2, decay, da, db;
  float one;                           // 1, where the compiler must not know it
};

// Eight consecutive elements as loaded: eight fp32, or eight bf16 in the first four words, or
// eight codes in the first two.
struct Raw8 {
  uint32_t w[8];
};

// The loads are not volatile: what is stored to a place depends on what was loaded from it, which
// orders the two, and nothing is loaded twice.
__device__ __forceinline__ void load8_f32(const float* p, int cnt, bool wide, Raw8& r) {
  if (wide && cnt == 8) {
    asm("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]),
          "=r"(r.w[6]), "=r"(r.w[7])
        : "l"(p));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = i < cnt ? __float_as_uint(p[i]) : 0u;
  }
}
__device__ __forceinline__ void load8_b16(const void* base, int cnt, bool wide, Raw8& r) {
  if (wide && cnt == 8) {
    const uint4 q = *static_cast<const uint4*>(base);
    r.w[0] = q.x, r.w[1] = q.y, r.w[2] = q.z, r.w[3] = q.w;
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i < cnt ? p[2 * i] : 0u;
      const uint32_t hi = 2 * i + 1 < cnt ? p[2 * i + 1] : 0u;
      r.w[i] = lo | (hi << 16);
    }
  }
}
__device__ __forceinline__ void load8_code(const uint8_t* p, int cnt, bool wide, uint2& q) {
  if (wide && cnt == 8) {
    q = *reinterpret_cast<const uint2*>(p);
  } else {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cnt) w[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
    q = make_uint2(w[0], w[1]);
  }
}
__device__ __forceinline__ void unpack8(const Raw8& r, bool bf16, float (&f)[8]) {
  if (bf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(r.w[i] << 16);
      f[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r.w[i]);
  }
}
__device__ __forceinline__ void store8_f32(float* p, int cnt, bool wide, const float (&f)[8]) {
  if (wide && cnt == 8) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]),
                 "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                 : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cnt) p[i] = f[i];
  }
}
__device__ __forceinline__ void store8_b16(__nv_bfloat16* p, int cnt, bool wide,
                                           const float (&f)[8]) {
  if (wide && cnt == 8) {
    uint4 q;
    uint32_t* u = reinterpret_cast<uint32_t*>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = q;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cnt) p[i] = __float2bfloat16_rn(f[i]);
  }
}
__device__ __forceinline__ void store8_code(uint8_t* p, int cnt, bool wide, uint2 q) {
  if (wide && cnt == 8) {
    *reinterpret_cast<uint2*>(p) = q;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cnt) p[i] = static_cast<uint8_t>((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
  }
}

// Three-way max that keeps a NaN (of magnitudes: max_abs3), and min.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void decode8(uint2 q, float scale, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? q.x : q.y;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(w >> (16 * (i & 1))), __NV_E4M3);
    const float2 v = mul2(__half22float2(__half2(h)), both(scale));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
__device__ __forceinline__ uint2 encode8(const float (&f)[8], float inv) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = __nv_cvt_float2_to_fp8x2(
        mul2(make_float2(f[2 * i], f[2 * i + 1]), both(inv)), __NV_SATFINITE, __NV_E4M3);
    w[i >> 1] |= c << (16 * (i & 1));
  }
  return make_uint2(w[0], w[1]);
}
// The largest magnitude of a warp's block of 256; a NaN stays one.  The maximum over the lanes is one
// of bit patterns: among non-negative values bit order is value order, NaN on top.
__device__ __forceinline__ float block_max(const float (&f)[8]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) top = max_abs3(top, f[i], f[i + 1]);
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
}
// amax times the rounded 1/448, as the format defines it (a division would cost more and differ by one
// unit of the last place at most), or 0 where that is below 2^-126: its reciprocal has to be finite.
__device__ __forceinline__ float scale_of(float amax) {
  const float scale = amax * (1.f / 448.f);
  return scale < 1.17549435e-38f ? 0.f : scale;
}

// One step of 8 elements: m, v and w in place; r = sqrt(v).  m and v take the definition's own
// roundings (each product and sum one), two values to an instruction, so that an 8-bit state does
// not depend on how they were computed.  The root and the reciprocal are the hardware's
// approximations (within 2 units of the last place): the exact ones cost 60 of 120 instructions for
// an element of 8-bit states, where the instructions bound the step.
__device__ __forceinline__ void adam8(const AdamScalars& a, const float (&grad)[8], float (&m)[8],
                                      float (&v)[8], float (&r)[8], float (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 g = mul2(make_float2(grad[i], grad[i + 1]), both(a.gs));
    // a sum as x 1 + y: two products and a packed add came out as a product and a fused one
    const float2 mm = fma2(mul2(both(a.b1), make_float2(m[i], m[i + 1])), both(a.one),
                           mul2(both(a.c1), g));
    const float2 vv = fma2(mul2(both(a.b2), make_float2(v[i], v[i + 1])), both(a.one),
                           mul2(both(a.c2), mul2(g, g)));
    m[i] = mm.x, m[i + 1] = mm.y;
    v[i] = vv.x, v[i + 1] = vv.y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r[i]) : "f"(vv.x));
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r[i + 1]) : "f"(vv.y));
    const float2 d = fma2(make_float2(r[i], r[i + 1]), both(a.da), both(a.db));
    float2 inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv.y) : "f"(d.y));
    const float2 ww = fma2(make_float2(w[i], w[i + 1]), both(a.decay), mul2(mm, inv));
    w[i] = ww.x, w[i + 1] = ww.y;
  }
}
// m and v of 8-bit states.
__device__ __forceinline__ void decode_states(uint2 qm, uint2 qr, float ms, float rs, float (&m)[8],
                                              float (&v)[8]) {
  decode8(qm, ms, m);
  decode8(qr, rs, v);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 r = make_float2(v[i], v[i + 1]), vv = mul2(r, r);
    v[i] = vv.x, v[i + 1] = vv.y;
  }
}

// The new codes and scales of a warp's block from m, v and the approximate r = sqrt(v).  A code is
// the nearest to x / scale, and r > 0 has at least the smallest code, 2^-9.  The quotient through the
// approximate root and reciprocal is off by less than 2^-21 of itself (root 2^-23 and the rounding of
// the exact one, reciprocal 2^-23, products 2^-24 each).  Where the codes of both ends of that
// interval differ, about one block in 200, or an r is below the smallest code, the lane takes the
// exact root and quotients.
__device__ __forceinline__ void encode_states(const float (&m)[8], const float (&v)[8],
                                              const float (&r)[8], uint2& qm, uint2& qr, float& ms,
                                              float& rs) {
  ms = scale_of(block_max(m));
  rs = scale_of(sqrtf(block_max(v)));          // the root of the largest v is the largest r
  float mi, ri;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(mi) : "f"(ms));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ri) : "f"(rs));
  if (ms == 0.f) mi = 0.f;
  if (rs == 0.f) ri = 0.f;
  constexpr float kLow = 1.f - 0x1p-21f, kHigh = 1.f + 0x1p-21f;
  const float floor = rs * 0.001953125f;
  float least = r[0];
#pragma unroll
  for (int i = 0; i < 8; i += 2) least = min3(least, r[i], r[i + 1]);
  qm = encode8(m, mi * kLow);
  qr = encode8(r, ri * kLow);
  const uint2 hm = encode8(m, mi * kHigh), hr = encode8(r, ri * kHigh);
  if (((qm.x ^ hm.x) | (qm.y ^ hm.y) | (qr.x ^ hr.x) | (qr.y ^ hr.y)) != 0u || least < floor) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = ms != 0.f ? __fdiv_rn(m[i], ms) : 0.f;
    qm = encode8(q, 1.f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      q[i] = v[i] != 0.f && rs != 0.f            // the approximate root of a v below 2^-126 is 0
                 ? max_abs3(__fdiv_rn(__fsqrt_rn(v[i]), rs), 0.001953125f, 0.f)
                 : 0.f;
    qr = encode8(q, 1.f);
  }
}

// One tile of a tensor, as the copying thread hands it to the warps that use it: pointers at the
// tile's first element.
struct AdamTile {
  void* param;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* r_scale;
  float* master;
  int n;                               // elements; 0 ends the block's work
  uint8_t whole;                       // all of it is in the ring
  uint8_t wide, group, kind;           // kind: the bits below
};
constexpr int kTileParam16 = 1, kTileGrad16 = 2, kTileMaster = 4, kTileState8 = 8;

// A part of a tile that its tensor ends in, or with any alignment, straight from global memory.  Each warp
// takes 256 consecutive elements: one block of an 8-bit state.  Unaligned it loads and stores element by
// element: 77 M weights and gradients one element off take 568 us with fp32 states (292 aligned), 470
// with 8-bit states (132).
__device__ __forceinline__ void adamw_ragged(const AdamTile& T, const AdamScalars& a, int part) {
  const int tid = threadIdx.x, at = part * kAdamPart + 8 * tid, warp = at / kStateBlock;
  if (at - 8 * (tid & 31) >= T.n) return;              // a warp's 256 elements, or none
  const int cnt = min(max(T.n - at, 0), 8);
  const bool wide = T.wide, pb = T.kind & kTileParam16, gb = T.kind & kTileGrad16;
  Raw8 rw, rg;
  if (T.master != nullptr)
    load8_f32(T.master + at, cnt, wide, rw);
  else if (pb)
    load8_b16(static_cast<const uint16_t*>(T.param) + at, cnt, wide, rw);
  else
    load8_f32(static_cast<const float*>(T.param) + at, cnt, wide, rw);
  if (gb)
    load8_b16(static_cast<const uint16_t*>(T.grad) + at, cnt, wide, rg);
  else
    load8_f32(static_cast<const float*>(T.grad) + at, cnt, wide, rg);
  float w[8], g[8], m[8], v[8], r[8];
  if (T.kind & kTileState8) {
    uint8_t* mc = static_cast<uint8_t*>(T.m) + at;
    uint8_t* rc = static_cast<uint8_t*>(T.v) + at;
    uint2 qm, qr;
    load8_code(mc, cnt, wide, qm);
    load8_code(rc, cnt, wide, qr);
    decode_states(qm, qr, T.m_scale[warp], T.r_scale[warp], m, v);
    unpack8(rw, pb && T.master == nullptr, w);
    unpack8(rg, gb, g);
    adam8(a, g, m, v, r, w);
    float ms, rs;
    encode_states(m, v, r, qm, qr, ms, rs);
    store8_code(mc, cnt, wide, qm);
    store8_code(rc, cnt, wide, qr);
    if ((tid & 31) == 0) {
      T.m_scale[warp] = ms;
      T.r_scale[warp] = rs;
    }
  } else {
    float* mp = static_cast<float*>(T.m) + at;
    float* vp = static_cast<float*>(T.v) + at;
    Raw8 rm, rv;
    load8_f32(mp, cnt, wide, rm);
    load8_f32(vp, cnt, wide, rv);
    unpack8(rm, false, m);
    unpack8(rv, false, v);
    unpack8(rw, pb && T.master == nullptr, w);
    unpack8(rg, gb, g);
    adam8(a, g, m, v, r, w);
    store8_f32(mp, cnt, wide, m);
    store8_f32(vp, cnt, wide, v);
  }
  if (T.master != nullptr) store8_f32(T.master + at, cnt, wide, w);
  if (pb)
    store8_b16(static_cast<__nv_bfloat16*>(T.param) + at, cnt, wide, w);
  else
    store8_f32(static_cast<float*>(T.param) + at, cnt, wide, w);
}

// The tensor that `chunk` belongs to, the last of `first` not behind it, from `at` on.  A warp looks
// at 32 entries at a time: one after the other, each a load that the next waits for, 38 tensors took
// 3 us.
__device__ __forceinline__ int find_tensor(const uint32_t* first, int count, uint32_t chunk,
                                           int at) {
  const int lane = threadIdx.x & 31;
  for (;;) {
    const int i = at + 1 + lane;
    const uint32_t not_behind = __ballot_sync(0xffffffffu, i < count && first[i] <= chunk);
    at += __popc(not_behind);
    if (not_behind != 0xffffffffu) return at;
  }
}

// ------------------------------------------------------------------ the walk over the tiles
// A warp of its own walks over the block's tiles, hands each to the other warps, and brings the
// whole ones into shared memory, ahead of their use by as many tiles as the ring has stages (long
// tiles: two with 8-bit states, one where a tensor of the launch has fp32 states): the elements by
// bulk copies, the scales, which may lie at any multiple of 4 bytes, by a copy of each.  What is in
// flight does not depend on the
// registers of the warps that compute, and neither the copies nor the descriptors cost them
// instructions.
__device__ __forceinline__ void scale_load(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on the barrier when this thread's copies before it are done.
__device__ __forceinline__ void scale_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

struct AdamRing {
  uint64_t* full;
  uint64_t* empty;
  AdamTile* tiles;
  uint8_t* data;
  uint32_t stage, parity;              // the next tile's place, and which turn of the ring
  __device__ __forceinline__ void next(uint32_t stages) {
    if (++stage == stages) stage = 0, parity ^= 1u;
  }
};

template <typename Args>
__device__ __forceinline__ void adamw_produce(const Args& args, AdamRing ring, bool skip) {
  constexpr int kTile = Args::kTile, kChunk = Args::kChunk;
  const int lane = threadIdx.x & 31;
  uint32_t issued = 0;
  int at = 0;                          // the tensor of the chunk
  const uint32_t data = smem_u32(ring.data);
  for (uint32_t chunk = blockIdx.x;; chunk += gridDim.x) {
    const bool end = chunk >= args.chunks;
    if (!end) at = find_tensor(args.first, args.count, chunk, at);
    const AdamTensor T = args.t[at];
    const long long start = end ? 0 : static_cast<long long>(chunk - args.first[at]) * kChunk;
    int left = end ? 0 : static_cast<int>(min(T.n - start, static_cast<long long>(kChunk)));
    const uint32_t nw = T.master != nullptr || !T.param_bf16 ? 4 : 2, ng = T.grad_bf16 ? 2 : 4,
                   ns = T.state8 ? 1 : 4, np = T.param_bf16 ? 2 : 4;
    AdamTile tile;
    tile.param = static_cast<uint8_t*>(T.param) + start * np;
    tile.grad = static_cast<const uint8_t*>(T.grad) + start * ng;
    tile.m = static_cast<uint8_t*>(T.m) + start * ns;
    tile.v = static_cast<uint8_t*>(T.v) + start * ns;
    tile.m_scale = T.m_scale + start / kStateBlock;
    tile.r_scale = T.r_scale + start / kStateBlock;
    tile.master = T.master != nullptr ? T.master + start : nullptr;
    tile.wide = T.wide;
    tile.group = T.group;
    tile.kind = (T.param_bf16 ? kTileParam16 : 0) | (T.grad_bf16 ? kTileGrad16 : 0) |
                (T.master != nullptr ? kTileMaster : 0) | (T.state8 ? kTileState8 : 0);
    do {
      // the place's turn before has been read (in the first turn it is free)
      if (issued >= args.stages) {
        bool ok = false;
        if (lane == 0 && !skip)
          ok = mbar_wait_bounded(&ring.empty[ring.stage], ring.parity ^ 1u, args.ticket + 1,
                                 kAdamWaitNs);
        if (!__shfl_sync(0xffffffffu, ok, 0)) goto drain;
      }
      tile.n = left < kTile ? left : kTile;
      tile.whole = T.wide && left >= kTile;
      ++issued;
      const uint32_t bar = smem_u32(&ring.full[ring.stage]);
      const uint32_t to = data + ring.stage * args.stage;
      if (lane == 0) {
        ring.tiles[ring.stage] = tile;
        if (tile.whole) {
          mbar_arrive_expect_tx(&ring.full[ring.stage], kTile * (nw + ng + 2 * ns));
          bulk_load(to, T.master != nullptr ? tile.master : tile.param, kTile * nw, bar);
          bulk_load(to + args.at_g, tile.grad, kTile * ng, bar);
          bulk_load(to + args.at_m, tile.m, kTile * ns, bar);
          bulk_load(to + args.at_v, tile.v, kTile * ns, bar);
        } else {
          mbar_arrive(&ring.full[ring.stage]);
        }
      }
      if (lane < Args::kScales) {
        constexpr int half = Args::kScales / 2;
        if (tile.whole && T.state8)
          scale_load(to + args.at_scales + 4 * lane,
                     lane < half ? tile.m_scale + lane : tile.r_scale + (lane - half));
        scale_arrive(bar);
      }
      ring.next(args.stages);
      left -= kTile;
      tile.param = static_cast<uint8_t*>(tile.param) + kTile * np;
      tile.grad = static_cast<const uint8_t*>(tile.grad) + kTile * ng;
      tile.m = static_cast<uint8_t*>(tile.m) + kTile * ns;
      tile.v = static_cast<uint8_t*>(tile.v) + kTile * ns;
      tile.m_scale += kTile / kStateBlock;
      tile.r_scale += kTile / kStateBlock;
      if (T.master != nullptr) tile.master += kTile;
    } while (left > 0);
    if (end) break;
  }
drain:
  // No copy may be in flight when the block ends: wait for the last turn's.
  for (uint32_t i = 0; i < (issued < args.stages ? issued : args.stages); ++i) {
    if (ring.stage == 0) ring.stage = args.stages, ring.parity ^= 1u;
    --ring.stage;
    mbar_wait_bounded(&ring.full[ring.stage], ring.parity, args.ticket + 1, kAdamWaitNs);
  }
}

// 8 fp32 or bf16 of this thread in a part of a stage.
__device__ __forceinline__ void ring8(const uint8_t* src, int part, bool bf16, float (&f)[8]) {
  Raw8 r;
  const uint4* p = reinterpret_cast<const uint4*>(src) +
                   (bf16 ? 1 : 2) * (part * kAdamThreads + threadIdx.x);
  const uint4 lo = p[0];
  r.w[0] = lo.x, r.w[1] = lo.y, r.w[2] = lo.z, r.w[3] = lo.w;
  if (!bf16) {
    const uint4 hi = p[1];
    r.w[4] = hi.x, r.w[5] = hi.y, r.w[6] = hi.z, r.w[7] = hi.w;
  }
  unpack8(r, bf16, f);
}

// A whole tile from its place in the ring.
template <bool PB, bool GB, bool MASTER, bool STATE8, typename Args>
__device__ __forceinline__ void adamw_whole(const Args& args, const AdamTile& T,
                                            const AdamScalars& a, const uint8_t* from,
                                            uint64_t* empty) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kBlocks = kAdamPart / kStateBlock;
  float* master = T.master + 8 * tid;
  uint8_t* param = static_cast<uint8_t*>(T.param) + (PB ? 16 : 32) * tid;
  uint8_t* mp = static_cast<uint8_t*>(T.m) + (STATE8 ? 8 : 32) * tid;
  uint8_t* vp = static_cast<uint8_t*>(T.v) + (STATE8 ? 8 : 32) * tid;
  float* m_scale = T.m_scale + warp;
  float* r_scale = T.r_scale + warp;
#pragma unroll
  for (int part = 0; part < Args::kParts; ++part) {
    const int at = part * kAdamPart;
    float w[8], g[8], m[8], v[8], r[8];
    ring8(from, part, PB && !MASTER, w);
    ring8(from + args.at_g, part, GB, g);
    if (STATE8) {
      const uint2 qm = *reinterpret_cast<const uint2*>(from + args.at_m + at + 8 * tid);
      const uint2 qr = *reinterpret_cast<const uint2*>(from + args.at_v + at + 8 * tid);
      const float* scales = reinterpret_cast<const float*>(from + args.at_scales) + warp;
      decode_states(qm, qr, scales[part * kBlocks], scales[(Args::kParts + part) * kBlocks], m, v);
    } else {
      ring8(from + args.at_m, part, false, m);
      ring8(from + args.at_v, part, false, v);
    }
    if (part + 1 == Args::kParts) {
      __syncwarp();
      if (lane == 0) mbar_arrive(empty);                   // the warp has read its part
    }
    adam8(a, g, m, v, r, w);
    if (MASTER) store8_f32(master + at, 8, true, w);
    if (PB)
      store8_b16(reinterpret_cast<__nv_bfloat16*>(param) + at, 8, true, w);
    else
      store8_f32(reinterpret_cast<float*>(param) + at, 8, true, w);
    if (STATE8) {
      uint2 qm, qr;
      float ms, rs;
      encode_states(m, v, r, qm, qr, ms, rs);
      store8_code(mp + at, 8, true, qm);
      store8_code(vp + at, 8, true, qr);
      if (lane == 0) {
        m_scale[part * kBlocks] = ms;
        r_scale[part * kBlocks] = rs;
      }
    } else {
      store8_f32(reinterpret_cast<float*>(mp) + at, 8, true, m);
      store8_f32(reinterpret_cast<float*>(vp) + at, 8, true, v);
    }
  }
}

// The warps that compute.
template <typename Args>
__device__ __forceinline__ void adamw_consume(const Args& args, const AdamScalars* groups,
                                              AdamRing ring) {
  const uint32_t stages = args.stages, bytes = args.stage;
  for (;;) {
    uint64_t* empty = &ring.empty[ring.stage];
    if (!mbar_wait_bounded(&ring.full[ring.stage], ring.parity, args.ticket + 1, kAdamWaitNs))
      return;
    const AdamTile& T = ring.tiles[ring.stage];
    if (T.n == 0) return;
    const AdamScalars a = groups[T.group];
    const uint8_t* from = ring.data + ring.stage * bytes;
    if (T.whole) {
      switch (T.kind) {
#define FLCE_ADAMW_KIND(k)                                                                      \
  case k:                                                                                       \
    adamw_whole<(k & kTileParam16) != 0, (k & kTileGrad16) != 0, (k & kTileMaster) != 0,        \
                (k & kTileState8) != 0>(args, T, a, from, empty);                               \
    break
        FLCE_ADAMW_KIND(0);
        FLCE_ADAMW_KIND(1);
        FLCE_ADAMW_KIND(2);
        FLCE_ADAMW_KIND(3);
        FLCE_ADAMW_KIND(5);
        FLCE_ADAMW_KIND(7);
        FLCE_ADAMW_KIND(8);
        FLCE_ADAMW_KIND(9);
        FLCE_ADAMW_KIND(10);
        FLCE_ADAMW_KIND(11);
        FLCE_ADAMW_KIND(13);
        FLCE_ADAMW_KIND(15);
#undef FLCE_ADAMW_KIND
      }
    } else {
#pragma unroll 1
      for (int part = 0; part < Args::kParts; ++part) adamw_ragged(T, a, part);
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(empty);
    }
    ring.next(stages);
  }
}

template <typename Args>
__global__ void __launch_bounds__(kAdamThreads + 32, kAdamBlocks) adamw_kernel(
    const __grid_constant__ Args args) {
  extern __shared__ __align__(128) uint8_t s_stages[];
  __shared__ uint64_t s_full[kAdamStages], s_empty[kAdamStages];
  __shared__ AdamTile s_tiles[kAdamStages];
  __shared__ AdamScalars s_group[kAdamGroups];
  __shared__ uint32_t s_rank;
  const int tid = threadIdx.x;
  const AdamRing ring{s_full, s_empty, s_tiles, s_stages, 0, 0};
  const float gscale = args.grad_scale != nullptr ? *args.grad_scale : 1.f;
  const bool skip = args.skip_nonfinite && !isfinite(gscale);
  if (tid >= kAdamThreads) {
    // the first copies are on their way while the other warps form the scalars
    if (tid == kAdamThreads) {
      for (uint32_t i = 0; i < args.stages; ++i) {
        mbar_init(&s_full[i], 1 + Args::kScales);
        mbar_init(&s_empty[i], kAdamThreads / 32);
      }
      fence_barrier_init();
    }
    __syncwarp();
    asm volatile("bar.arrive 1, %0;" ::"n"(kAdamThreads + 32) : "memory");
    adamw_produce(args, ring, skip);
  } else {
    if (tid < args.groups) {
      const AdamGroup& g = args.g[tid];
      // t log beta in 64 bits, everything after it in fp32: a thread's 64-bit expm1 held a block
      // back by 3 us
      const double t = static_cast<double>(*args.step + 1);
      const float lr = g.lr_device != nullptr ? *g.lr_device : g.lr;
      const float size = lr / expm1f(static_cast<float>(t * g.log_beta1));   // beta1^t - 1
      AdamScalars a;
      a.gs = gscale;
      a.b1 = g.beta1;
      a.c1 = g.c1;
      a.b2 = g.beta2;
      a.c2 = g.c2;
      a.one = g.one;
      a.decay = 1.f - lr * g.weight_decay;
      a.da = 1.f / (size * sqrtf(-expm1f(static_cast<float>(t * g.log_beta2))));
      a.db = g.eps / size;
      // a rate of 0 (or too small to divide by): the reciprocal flushes to 0 and nothing moves
      if (fabsf(size) < 1e-30f) a.da = a.db = 1e38f;
      s_group[tid] = a;
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kAdamThreads + 32) : "memory");
    if (!skip) adamw_consume(args, s_group, ring);
  }
  // The block that arrives last has seen every other block read *step: it counts the step and
  // leaves the ticket zero for the next call.
  if (!args.last) return;
  __syncthreads();
  if (tid == 0) s_rank = atomicAdd(args.ticket, 1u);
  __syncthreads();
  if (tid == 0 && s_rank == gridDim.x - 1) {
    if (!skip) *args.step += 1;
    *args.ticket = 0u;
  }
}

// ------------------------------------------------------------------------------ gradient norm
struct NormTensor {
  const void* grad;
  long long n;
  uint8_t bf16, wide, pad[6];
};
template <int N>
struct NormArgs {
  uint32_t first[N];
  NormTensor t[N];
  int count;
  uint32_t chunks;
  double* partial;                     // one sum for each block
};

static_assert(sizeof(NormArgs<kNormTensors>) <= 32764, "a launch's parameters");

// A block's sum of 64-bit values, in a fixed order; valid in thread 0.
__device__ __forceinline__ double norm_block_sum(double v, double (&s_sum)[kNormThreads / 32]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kNormThreads / 32; ++w) v += s_sum[w];
  return v;
}

// A thread's 64 squares of a whole aligned chunk, four 32-byte loads in flight.
template <bool BF16>
__device__ __forceinline__ float norm_chunk(const void* grad, long long start) {
  constexpr int PER = BF16 ? 16 : 8;                       // elements of a load
  const uint8_t* p = static_cast<const uint8_t*>(grad) + (start / PER + threadIdx.x) * 32;
  float acc = 0.f;
#pragma unroll
  for (int pass = 0; pass < kNormChunk / (PER * kNormThreads); pass += 4) {
    Raw8 r[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      load8_f32(reinterpret_cast<const float*>(p + (pass + u) * (32 * kNormThreads)), 8, true, r[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (BF16) {
          const float lo = __uint_as_float(r[u].w[i] << 16);
          const float hi = __uint_as_float(r[u].w[i] & 0xffff0000u);
          acc = fmaf(lo, lo, acc);
          acc = fmaf(hi, hi, acc);
        } else {
          const float f = __uint_as_float(r[u].w[i]);
          acc = fmaf(f, f, acc);
        }
      }
  }
  return acc;
}
// The same of a chunk that the tensor ends in, or with any alignment (element by element: 236 M bf16
// values one element off take 160 us, 75 aligned).
__device__ __forceinline__ float norm_ragged(const NormTensor& T, long long start) {
  float acc = 0.f;
#pragma unroll 1
  for (int pass = 0; pass < kNormChunk / (8 * kNormThreads); ++pass) {
    const long long at = start + (pass * kNormThreads + threadIdx.x) * 8;
    const long long left = T.n - at;
    if (left <= 0) break;
    const int cnt = left >= 8 ? 8 : static_cast<int>(left);
    Raw8 r;
    float f[8];
    if (T.bf16)
      load8_b16(static_cast<const uint16_t*>(T.grad) + at, cnt, T.wide, r);
    else
      load8_f32(static_cast<const float*>(T.grad) + at, cnt, T.wide, r);
    unpack8(r, T.bf16, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc = fmaf(f[i], f[i], acc);
  }
  return acc;
}

template <int N>
__global__ void __launch_bounds__(kNormThreads) grad_norm_kernel(
    const __grid_constant__ NormArgs<N> args) {
  __shared__ double s_sum[kNormThreads / 32];
  // the sum over the blocks may be made ready to start (it waits for this launch's end)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  double sum = 0.0;
  int tensor = 0;                      // of the block's chunk
  for (uint32_t chunk = blockIdx.x; chunk < args.chunks; chunk += gridDim.x) {
    tensor = find_tensor(args.first, args.count, chunk, tensor);
    const NormTensor& T = args.t[tensor];
    const long long start = static_cast<long long>(chunk - args.first[tensor]) * kNormChunk;
    float acc = 0.f;
    if (!T.wide || start + kNormChunk > T.n)
      acc = norm_ragged(T, start);
    else if (T.bf16)
      acc = norm_chunk<true>(T.grad, start);
    else
      acc = norm_chunk<false>(T.grad, start);
    sum += static_cast<double>(acc);
  }
  sum = norm_block_sum(sum, s_sum);
  if (tid == 0) args.partial[blockIdx.x] = sum;
}

// The launch before still writes the partials while this one starts, so they are no read-only data
// of this kernel: no __restrict__, and loads from L2 (__ldcg) behind the wait.
__global__ void __launch_bounds__(kNormThreads) grad_norm_finish_kernel(
    const double* partial, long long parts, float max_norm, float* norm_out, float* factor_out) {
  __shared__ double s_sum[kNormThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");       // the partials are complete
  double sum = 0.0;
  for (long long i = threadIdx.x; i < parts; i += kNormThreads)
    sum += __ldcg(partial + i);
  sum = norm_block_sum(sum, s_sum);
  if (threadIdx.x != 0) return;
  const float norm = static_cast<float>(sqrt(sum));
  *norm_out = norm;
  if (factor_out != nullptr)
    *factor_out = isfinite(norm) ? fminf(1.f, max_norm / (norm + 1e-6f)) : __int_as_float(0x7fffffff);
}

}  // namespace flce
