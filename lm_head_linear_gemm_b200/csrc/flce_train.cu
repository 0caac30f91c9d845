// C ABI of the training-step operators around the head (include/flce_train.h): argument checks
// and launches.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "../../include/flce_train.h"
#include "host.h"
#include "optim.cuh"
#include "qk_norm.cuh"

using namespace flce;

namespace {

#define FLCE_TRY(expr)              \
  do {                              \
    const int _rc = (expr);         \
    if (_rc != FLCE_OK) return _rc; \
  } while (0)

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int launched() {
  count_launch();
  return cudaGetLastError() == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

// A call's elements: their chunks fit 32 bits in one launch.
constexpr int64_t kMaxElements = int64_t(1) << 42;

// Lets a kernel have more dynamic shared memory than a launch gets unasked.  The attribute belongs to
// the device: set once for each, `done` has their bits.
int allow_shared(const void* kernel, int bytes, int device, std::atomic<uint64_t>* done) {
  const uint64_t bit = uint64_t(1) << device;
  if (done->load(std::memory_order_relaxed) & bit) return FLCE_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess)
    return FLCE_ERR_CUDA;
  done->fetch_or(bit, std::memory_order_relaxed);
  return FLCE_OK;
}

// Launches a kernel that waits (griddepcontrol.wait) for the one before it on the stream: it may be
// brought onto the GPU while that one still runs.
template <typename... P, typename... A>
int launch_after(void (*kernel)(P...), int grid, dim3 block, cudaStream_t st, A... args) {
  cudaLaunchConfig_t config{};
  config.gridDim = dim3(grid);
  config.blockDim = block;
  config.stream = st;
  cudaLaunchAttribute attribute{};
  attribute.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attribute.val.programmaticStreamSerializationAllowed = 1;
  config.attrs = &attribute;
  config.numAttrs = 1;
  const bool ok = cudaLaunchKernelEx(&config, kernel, static_cast<P>(args)...) == cudaSuccess;
  const int rc = launched();
  return ok ? rc : FLCE_ERR_CUDA;
}

bool dtype_ok(int32_t t) { return t == FLCE_DTYPE_F32 || t == FLCE_DTYPE_BF16; }
int64_t dtype_bytes(int32_t t) { return t == FLCE_DTYPE_BF16 ? 2 : 4; }

// ------------------------------------------------------------------------------ query / key norm
int qk_shape_ok(const flce_qk_shape* s) {
  if (s == nullptr || s->B < 0 || s->T < 0 || s->Hq < 0 || s->Hk < 0 || s->Hq > 4096 ||
      s->Hk > 4096 || s->D < 16 || s->D > 512 || s->rot < 0 || s->rot > s->D ||
      !(s->eps >= 0.f) || !dtype_ok(s->dtype) || !dtype_ok(s->gamma_dtype) ||
      (s->interleaved != 0 && s->interleaved != 1))
    return FLCE_ERR_ARG;
  if (s->D % 16 != 0 || s->rot % 16 != 0) return FLCE_ERR_ALIGN;
  if (s->B > 0 && s->T > 0x7fffffffll / s->B) return FLCE_ERR_ARG;
  return FLCE_OK;
}

// Two arrays of n floats that share an element; NULL shares none.
bool floats_overlap(const float* a, const float* b, int64_t n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  const uintptr_t bytes = static_cast<uintptr_t>(n) * sizeof(float);
  return a != nullptr && b != nullptr && (x < y ? y - x : x - y) < bytes;
}

// A view of H heads: alignment, and for a written one that no two elements share a place.
int qk_view_ok(const flce_qk_shape* s, const flce_qk_view* v, int64_t H, bool written) {
  if (v == nullptr) return H == 0 ? FLCE_OK : FLCE_ERR_ARG;
  if (s->B * s->T * H == 0) return FLCE_OK;
  if (v->ptr == nullptr) return FLCE_ERR_ARG;
  if (!aligned(v->ptr, 16)) return FLCE_ERR_ALIGN;
  const int64_t size[3] = {s->B, s->T, H}, stride[3] = {v->batch, v->token, v->head};
  const int64_t unit = 16 / dtype_bytes(s->dtype);
  int order[3], n = 0;
  for (int i = 0; i < 3; ++i) {
    if (size[i] <= 1) continue;
    if (stride[i] < 0 || stride[i] > (int64_t(1) << 40)) return FLCE_ERR_ARG;
    if (stride[i] % unit != 0) return FLCE_ERR_ALIGN;
    int at = n++;
    for (; at > 0 && stride[order[at - 1]] > stride[i]; --at) order[at] = order[at - 1];
    order[at] = i;
  }
  __int128 extent = s->D;              // elements the inner dimensions span
  for (int i = 0; written && i < n; ++i) {
    if (stride[order[i]] < extent) return FLCE_ERR_ARG;
    extent += static_cast<__int128>(stride[order[i]]) * (size[order[i]] - 1);
  }
  return FLCE_OK;
}

int qk_common_ok(const flce_qk_shape* s, const void* gamma_q, const void* gamma_k,
                 const float* inv_freq, const int64_t* positions) {
  FLCE_TRY(qk_shape_ok(s));
  if (s->rot > 0 && inv_freq == nullptr) return FLCE_ERR_ARG;
  if (!aligned(gamma_q, 16) || !aligned(gamma_k, 16) || !aligned(inv_freq, 4) ||
      !aligned(positions, 8))
    return FLCE_ERR_ALIGN;
  return FLCE_OK;
}

QkDivisor qk_divisor(int64_t d) {
  QkDivisor q{static_cast<uint32_t>(d), 0, 31};
  while ((int64_t(1) << (q.shift - 31)) < d) ++q.shift;
  const uint64_t one = uint64_t(1) << q.shift;
  q.mul = static_cast<uint32_t>((one + q.d - 1) / q.d);
  return q;
}

QkView qk_view(const flce_qk_view* v) {
  return v == nullptr ? QkView{} : QkView{v->ptr, v->batch, v->token, v->head};
}

QkArgs qk_args(const flce_qk_shape* s, const flce_qk_view* q, const flce_qk_view* k,
               const void* gamma_q, const void* gamma_k, const float* inv_freq,
               const int64_t* positions, int64_t positions_batch, int lanes, int sms, int blocks) {
  QkArgs a{};
  a.q = qk_view(q);
  a.k = qk_view(k);
  a.gamma_q = gamma_q;
  a.gamma_k = gamma_k;
  a.inv_freq = inv_freq;
  a.positions = reinterpret_cast<const long long*>(positions);
  a.positions_batch = positions_batch;
  a.T = qk_divisor(s->T);
  a.Hq = static_cast<int>(s->Hq);
  a.Hk = static_cast<int>(s->Hk);
  a.D = static_cast<int>(s->D);
  a.rot = static_cast<int>(s->rot);
  a.eps = s->eps;
  a.gamma_f32 = s->gamma_dtype == FLCE_DTYPE_F32;
  // A warp takes the passes (rows of 32 / lanes heads) of a whole token, or a segment of them: as
  // many segments as make the busiest warp's share the least.  A token's angles count as one more
  // pass of each segment.
  const int64_t tokens = s->B * s->T, rows = 32 / lanes;
  const int64_t passes = (s->Hq + rows - 1) / rows + (s->Hk + rows - 1) / rows;
  const int64_t warps = static_cast<int64_t>(blocks) * sms * kQkWarps;
  int64_t best = passes, least = INT64_MAX;
  for (int64_t n = 1; n <= passes && n <= 64; ++n) {
    const int64_t each = (passes + n - 1) / n;
    const int64_t cost = (tokens * ((passes + each - 1) / each) + warps - 1) / warps * (each + 1);
    if (cost < least) least = cost, best = each;
    if (tokens * n > 64 * warps) break;             // fine enough
  }
  a.seg_passes = static_cast<uint32_t>(best);
  a.segs = qk_divisor((passes + best - 1) / best);
  a.items = static_cast<uint32_t>(tokens * a.segs.d);
  return a;
}

// Lanes of a row: its 16-element units, or the next number of lanes that gives a warp as many rows.
// Groups of 3, 5, 6 and 10 lanes take 10, 6, 5 and 3 rows of heads of 48, 80, 96 and 160 where the
// next power of two takes 8, 4, 4 and 2 (4911 tokens of 20 heads of 80, fp32: 21.3 -> 18.1 us).
int qk_lanes(int64_t D) {
  const int units = static_cast<int>(D / 16);
  return units <= 6 ? units : units <= 8 ? 8 : units <= 10 ? 10 : units <= 16 ? 16 : 32;
}

template <typename T, int LANES, bool INTER, bool BWD>
int qk_launch(const QkArgs& a, int device, int grid, cudaStream_t st) {
  constexpr int bytes = QkRing<T, BWD>::kBytes;
  auto kernel = qk_norm_rope_kernel<T, LANES, INTER, BWD>;
  static std::atomic<uint64_t> done{0};
  FLCE_TRY(allow_shared(reinterpret_cast<const void*>(kernel), bytes, device, &done));
  kernel<<<grid, 32 * kQkWarps, bytes, st>>>(a);
  return launched();
}

template <typename T, bool INTER, bool BWD>
int qk_launch_lanes(int lanes, const QkArgs& a, int device, int grid, cudaStream_t st) {
  switch (lanes) {
    case 1: return qk_launch<T, 1, INTER, BWD>(a, device, grid, st);
    case 2: return qk_launch<T, 2, INTER, BWD>(a, device, grid, st);
    case 3: return qk_launch<T, 3, INTER, BWD>(a, device, grid, st);
    case 4: return qk_launch<T, 4, INTER, BWD>(a, device, grid, st);
    case 5: return qk_launch<T, 5, INTER, BWD>(a, device, grid, st);
    case 6: return qk_launch<T, 6, INTER, BWD>(a, device, grid, st);
    case 8: return qk_launch<T, 8, INTER, BWD>(a, device, grid, st);
    case 10: return qk_launch<T, 10, INTER, BWD>(a, device, grid, st);
    case 16: return qk_launch<T, 16, INTER, BWD>(a, device, grid, st);
    default: return qk_launch<T, 32, INTER, BWD>(a, device, grid, st);
  }
}

template <bool BWD>
int qk_run(const flce_qk_shape* s, int lanes, const QkArgs& a, int device, int grid,
           cudaStream_t st) {
  const bool inter = s->interleaved != 0;
  if (s->dtype == FLCE_DTYPE_BF16)
    return inter ? qk_launch_lanes<__nv_bfloat16, true, BWD>(lanes, a, device, grid, st)
                 : qk_launch_lanes<__nv_bfloat16, false, BWD>(lanes, a, device, grid, st);
  return inter ? qk_launch_lanes<float, true, BWD>(lanes, a, device, grid, st)
               : qk_launch_lanes<float, false, BWD>(lanes, a, device, grid, st);
}

// Blocks of a launch: persistent ones that fill the GPU, fewer when there are fewer items.
int qk_grid(const QkArgs& a, int blocks, int sms) {
  const int64_t need = (static_cast<int64_t>(a.items) + kQkWarps - 1) / kQkWarps;
  const int64_t most = static_cast<int64_t>(blocks) * sms;
  return static_cast<int>(need < most ? need : most);
}

// ------------------------------------------------------------------------------ AdamW
int adamw_tensor_ok(const flce_adamw_tensor& t, const void* grad, int n_groups) {
  if (t.n < 0 || !dtype_ok(t.param_dtype) || !dtype_ok(t.grad_dtype) || t.group < 0 ||
      t.group >= n_groups || (t.state != FLCE_STATE_F32 && t.state != FLCE_STATE_E4M3) ||
      t.n > kMaxElements)
    return FLCE_ERR_ARG;
  if (t.n == 0 || grad == nullptr) return FLCE_OK;
  const bool eight = t.state == FLCE_STATE_E4M3;
  if (t.param == nullptr || t.m == nullptr || t.v == nullptr ||
      (eight && (t.m_scale == nullptr || t.r_scale == nullptr)) ||
      (t.master != nullptr && t.param_dtype != FLCE_DTYPE_BF16))
    return FLCE_ERR_ARG;
  if (!aligned(t.param, dtype_bytes(t.param_dtype)) || !aligned(grad, dtype_bytes(t.grad_dtype)) ||
      (!eight && (!aligned(t.m, 4) || !aligned(t.v, 4))) || !aligned(t.m_scale, 4) ||
      !aligned(t.r_scale, 4) || !aligned(t.master, 4))
    return FLCE_ERR_ALIGN;
  return FLCE_OK;
}

bool wide_ok(const void* p, int32_t dtype) {
  return aligned(p, dtype == FLCE_DTYPE_BF16 ? 16 : 32);
}

AdamTensor adamw_tensor(const flce_adamw_tensor& t, const void* grad) {
  const bool eight = t.state == FLCE_STATE_E4M3;
  AdamTensor o{};
  o.param = t.param;
  o.grad = grad;
  o.m = t.m;
  o.v = t.v;
  o.m_scale = t.m_scale;
  o.r_scale = t.r_scale;
  o.master = t.master;
  o.n = t.n;
  o.param_bf16 = t.param_dtype == FLCE_DTYPE_BF16;
  o.grad_bf16 = t.grad_dtype == FLCE_DTYPE_BF16;
  o.state8 = eight;
  o.group = static_cast<uint8_t>(t.group);
  o.wide = wide_ok(t.param, t.param_dtype) && wide_ok(grad, t.grad_dtype) &&
           aligned(t.m, eight ? 16 : 32) && aligned(t.v, eight ? 16 : 32) &&
           aligned(t.master, 32);
  return o;
}

// The root takes a v below 2^-126 for 0: the smallest eps that keeps m / eps near 1 there.
constexpr double kMinEps = 1.0 / (1ull << 60);

AdamGroup adamw_group(const flce_adamw_group& g) {
  AdamGroup o{};
  o.lr_device = g.lr_device;
  o.log_beta1 = std::log(g.beta1);
  o.log_beta2 = std::log(g.beta2);
  o.lr = static_cast<float>(g.lr);
  o.beta1 = static_cast<float>(g.beta1);
  o.beta2 = static_cast<float>(g.beta2);
  o.c1 = static_cast<float>(1.0 - g.beta1);
  o.c2 = static_cast<float>(1.0 - g.beta2);
  o.one = 1.f;
  o.eps = static_cast<float>(g.eps);
  o.weight_decay = static_cast<float>(g.weight_decay);
  return o;
}

// A stage of the ring holds a tile of the launch's widest tensor; the ring as many stages as fit.  All
// tensors count, those too short or too unaligned to enter the ring among them: a norm's weights with
// fp32 states next to matrices in 8 bits leave one stage of two (77 M weights 132 -> 182 us, 236 M
// with master copies 635 -> 654).
template <typename Args>
void adamw_stage(Args* a) {
  constexpr int kTile = Args::kTile;
  uint32_t w = 2, g = 2, st = 1;
  for (int i = 0; i < a->count; ++i) {
    const AdamTensor& t = a->t[i];
    if (t.master != nullptr || !t.param_bf16) w = 4;
    if (!t.grad_bf16) g = 4;
    if (!t.state8) st = 4;
  }
  a->at_g = w * kTile;
  a->at_m = a->at_g + g * kTile;
  a->at_v = a->at_m + st * kTile;
  a->at_scales = a->at_v + st * kTile;
  a->stage = a->at_scales + Args::kScales * 4;
  a->stage = (a->stage + 127) / 128 * 128;
  a->stages = kAdamRing / a->stage;
  if (a->stages > kAdamStages) a->stages = kAdamStages;
}

struct AdamwCall {
  const flce_adamw_tensor* tensors;
  const void* const* grads;
  int64_t count;
  const flce_adamw_group* groups;
  int n_groups;
  const float* grad_scale;
  int64_t* step;
  int skip_nonfinite;
  void* scratch;
  cudaStream_t stream;
};

// A step's launches, for N tensors each.
template <int N, int PARTS>
int adamw_launches(const AdamwCall& c, int device, int sms) {
  using Args = AdamArgs<N, PARTS>;
  Args a;
  a.groups = c.n_groups;
  for (int i = 0; i < c.n_groups; ++i) a.g[i] = adamw_group(c.groups[i]);
  a.skip_nonfinite = c.skip_nonfinite ? 1 : 0;
  a.grad_scale = c.grad_scale;
  a.step = reinterpret_cast<long long*>(c.step);
  a.ticket = static_cast<uint32_t*>(c.scratch);
  static std::atomic<uint64_t> done{0};
  FLCE_TRY(
      allow_shared(reinterpret_cast<const void*>(adamw_kernel<Args>), kAdamRing, device, &done));
  int64_t next = 0;
  do {
    a.count = 0;
    int64_t chunks = 0;
    for (; next < c.count && a.count < N; ++next) {
      if (c.tensors[next].n == 0 || c.grads[next] == nullptr) continue;
      a.first[a.count] = static_cast<uint32_t>(chunks);
      a.t[a.count++] = adamw_tensor(c.tensors[next], c.grads[next]);
      chunks += (c.tensors[next].n + Args::kChunk - 1) / Args::kChunk;
    }
    if (a.count == 0) a.t[0] = AdamTensor{};
    a.chunks = static_cast<uint32_t>(chunks);
    a.last = next == c.count;
    adamw_stage(&a);
    const int64_t most = static_cast<int64_t>(kAdamBlocks) * sms;
    const int grid = static_cast<int>(chunks < 1 ? 1 : chunks < most ? chunks : most);
    adamw_kernel<Args><<<grid, kAdamThreads + 32, kAdamRing, c.stream>>>(a);
    FLCE_TRY(launched());
  } while (next < c.count);
  return FLCE_OK;
}

// The partial sums of a norm's launches, for N tensors each; *parts of them.
template <int N>
int norm_launches(const void* const* grads, const int64_t* sizes, const int32_t* dtypes,
                  int64_t count, double* partial, int sms, cudaStream_t st, int64_t* parts) {
  NormArgs<N> a;
  int64_t next = 0;
  *parts = 0;
  while (next < count) {
    a.count = 0;
    int64_t chunks = 0;
    for (; next < count && a.count < N; ++next) {
      if (sizes[next] == 0 || grads[next] == nullptr) continue;
      a.first[a.count] = static_cast<uint32_t>(chunks);
      NormTensor& t = a.t[a.count++];
      t.grad = grads[next];
      t.n = sizes[next];
      t.bf16 = dtypes[next] == FLCE_DTYPE_BF16;
      t.wide = aligned(grads[next], 32);
      chunks += (sizes[next] + kNormChunk - 1) / kNormChunk;
    }
    if (a.count == 0) break;           // the rest held no elements
    a.chunks = static_cast<uint32_t>(chunks);
    a.partial = partial + *parts;
    const int64_t most = 4ll * sms < kNormBlocks ? 4ll * sms : kNormBlocks;
    const int grid = static_cast<int>(chunks < most ? chunks : most);
    grad_norm_kernel<N><<<grid, kNormThreads, 0, st>>>(a);
    FLCE_TRY(launched());
    *parts += grid;
  }
  return FLCE_OK;
}

}  // namespace

extern "C" {

int flce_qk_norm_rope_forward(const flce_qk_shape* s, const flce_qk_view* q, const flce_qk_view* k,
                              const void* gamma_q, const void* gamma_k, const float* inv_freq,
                              const int64_t* positions, int64_t positions_batch,
                              const flce_qk_view* q_out, const flce_qk_view* k_out, void* stream) {
  FLCE_TRY(qk_common_ok(s, gamma_q, gamma_k, inv_freq, positions));
  FLCE_TRY(qk_view_ok(s, q, s->Hq, false));
  FLCE_TRY(qk_view_ok(s, k, s->Hk, false));
  FLCE_TRY(qk_view_ok(s, q_out, s->Hq, true));
  FLCE_TRY(qk_view_ok(s, k_out, s->Hk, true));
  int device = 0, sms = 0;
  FLCE_TRY(device_sms(&device, &sms));
  if (s->B * s->T * (s->Hq + s->Hk) == 0) return FLCE_OK;
  const int lanes = qk_lanes(s->D);
  QkArgs a = qk_args(s, q, k, gamma_q, gamma_k, inv_freq, positions, positions_batch, lanes, sms,
                     kQkBlocks);
  a.yq = qk_view(q_out);
  a.yk = qk_view(k_out);
  return qk_run<false>(s, lanes, a, device, qk_grid(a, kQkBlocks, sms),
                       static_cast<cudaStream_t>(stream));
}

size_t flce_qk_norm_rope_workspace_bytes(const flce_qk_shape* s) {
  if (qk_shape_ok(s) != FLCE_OK) return 0;
  return static_cast<size_t>(kQkMaxParts) * 2 * static_cast<size_t>(s->D) * sizeof(float);
}

int flce_qk_norm_rope_backward(const flce_qk_shape* s, const flce_qk_view* dq_out,
                               const flce_qk_view* dk_out, const flce_qk_view* q,
                               const flce_qk_view* k, const void* gamma_q, const void* gamma_k,
                               const float* inv_freq, const int64_t* positions,
                               int64_t positions_batch, const flce_qk_view* dq,
                               const flce_qk_view* dk, float* dgamma_q, float* dgamma_k,
                               int accumulate_dgamma, void* workspace, size_t workspace_bytes,
                               void* stream) {
  FLCE_TRY(qk_common_ok(s, gamma_q, gamma_k, inv_freq, positions));
  FLCE_TRY(qk_view_ok(s, dq_out, s->Hq, false));
  FLCE_TRY(qk_view_ok(s, dk_out, s->Hk, false));
  FLCE_TRY(qk_view_ok(s, q, s->Hq, false));
  FLCE_TRY(qk_view_ok(s, k, s->Hk, false));
  FLCE_TRY(qk_view_ok(s, dq, s->Hq, true));
  FLCE_TRY(qk_view_ok(s, dk, s->Hk, true));
  if (workspace == nullptr) return FLCE_ERR_ARG;
  if (!aligned(workspace, 256) || !aligned(dgamma_q, 4) || !aligned(dgamma_k, 4))
    return FLCE_ERR_ALIGN;
  if (workspace_bytes < flce_qk_norm_rope_workspace_bytes(s)) return FLCE_ERR_WORKSPACE;
  // the two sums are stored by different warps: in one place they would overwrite each other
  if (floats_overlap(dgamma_q, dgamma_k, s->D)) return FLCE_ERR_ARG;
  int device = 0, sms = 0;
  FLCE_TRY(device_sms(&device, &sms));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int lanes = qk_lanes(s->D);
  int grid = 0;
  if (s->B * s->T * (s->Hq + s->Hk) != 0) {
    // never more than the workspace has room for, whatever the device
    const int blocks = kQkBlocks * sms <= kQkMaxParts ? kQkBlocks : 1;
    if (blocks * sms > kQkMaxParts) return FLCE_ERR_DEVICE;
    QkArgs a = qk_args(s, q, k, gamma_q, gamma_k, inv_freq, positions, positions_batch, lanes, sms,
                       blocks);
    a.dq = qk_view(dq_out);
    a.dk = qk_view(dk_out);
    a.yq = qk_view(dq);
    a.yk = qk_view(dk);
    a.partial = static_cast<float*>(workspace);
    grid = qk_grid(a, blocks, sms);
    FLCE_TRY(qk_run<true>(s, lanes, a, device, grid, st));
  }
  if (dgamma_q == nullptr && dgamma_k == nullptr) return FLCE_OK;
  const int D = static_cast<int>(s->D);
  return launch_after(qk_dgamma_kernel, (2 * D + 31) / 32, dim3(32, 32), st,
                      static_cast<const float*>(workspace), grid, D, dgamma_q, dgamma_k,
                      accumulate_dgamma ? 1 : 0);
}

int flce_adamw_step(const flce_adamw_tensor* tensors, const void* const* grads, int64_t count,
                    const flce_adamw_group* groups, int n_groups, const float* grad_scale,
                    int64_t* step, int skip_nonfinite, void* scratch, void* stream) {
  if (count < 0 || (count > 0 && (tensors == nullptr || grads == nullptr)) || groups == nullptr ||
      n_groups < 1 || n_groups > FLCE_ADAMW_MAX_GROUPS || step == nullptr || scratch == nullptr)
    return FLCE_ERR_ARG;
  if (!aligned(grad_scale, 4) || !aligned(step, 8) || !aligned(scratch, 16)) return FLCE_ERR_ALIGN;
  for (int i = 0; i < n_groups; ++i) {
    const flce_adamw_group& g = groups[i];
    if (!(g.beta1 >= 0.0 && g.beta1 < 1.0) || !(g.beta2 >= 0.0 && g.beta2 < 1.0) ||
        !(g.eps >= kMinEps) || !std::isfinite(g.weight_decay) ||
        (g.lr_device == nullptr && !std::isfinite(g.lr)))
      return FLCE_ERR_ARG;
    if (!aligned(g.lr_device, 4)) return FLCE_ERR_ALIGN;
  }
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) {
    FLCE_TRY(adamw_tensor_ok(tensors[i], grads[i], n_groups));
    if ((total += tensors[i].n) > kMaxElements) return FLCE_ERR_ARG;
  }
  int device = 0, sms = 0;
  FLCE_TRY(device_sms(&device, &sms));
  const AdamwCall call{tensors, grads, count, groups, n_groups, grad_scale, step, skip_nonfinite,
                       scratch, static_cast<cudaStream_t>(stream)};
  // tiles of one step where the blocks have fewer than four of two
  const bool few = count <= kFewTensors,
             small = total < 4ll * kAdamBlocks * sms * AdamArgs<1, 2>::kTile;
  if (small)
    return few ? adamw_launches<kFewTensors, 1>(call, device, sms)
               : adamw_launches<kAdamTensors, 1>(call, device, sms);
  return few ? adamw_launches<kFewTensors, 2>(call, device, sms)
             : adamw_launches<kAdamTensors, 2>(call, device, sms);
}

size_t flce_grad_norm_workspace_bytes(int64_t count) {
  if (count < 0) return 0;
  const size_t launches = static_cast<size_t>(count / kNormTensors) + 1;
  return launches * kNormBlocks * sizeof(double);
}

int flce_grad_norm(const void* const* grads, const int64_t* sizes, const int32_t* dtypes,
                   int64_t count, float max_norm, float* norm, float* factor, void* workspace,
                   size_t workspace_bytes, void* stream) {
  if (count < 0 || (count > 0 && (grads == nullptr || sizes == nullptr || dtypes == nullptr)) ||
      norm == nullptr || workspace == nullptr || (factor != nullptr && !(max_norm >= 0.f)))
    return FLCE_ERR_ARG;
  if (!aligned(norm, 4) || !aligned(factor, 4) || !aligned(workspace, 256)) return FLCE_ERR_ALIGN;
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (sizes[i] < 0 || sizes[i] > kMaxElements || !dtype_ok(dtypes[i])) return FLCE_ERR_ARG;
    if ((total += sizes[i]) > kMaxElements) return FLCE_ERR_ARG;
    if (!aligned(grads[i], dtype_bytes(dtypes[i]))) return FLCE_ERR_ALIGN;
  }
  if (workspace_bytes < flce_grad_norm_workspace_bytes(count)) return FLCE_ERR_WORKSPACE;
  int device = 0, sms = 0;
  FLCE_TRY(device_sms(&device, &sms));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  double* partial = static_cast<double*>(workspace);
  int64_t parts = 0;
  if (count <= kFewTensors)
    FLCE_TRY(norm_launches<kFewTensors>(grads, sizes, dtypes, count, partial, sms, st, &parts));
  else
    FLCE_TRY(norm_launches<kNormTensors>(grads, sizes, dtypes, count, partial, sms, st, &parts));
  return launch_after(grad_norm_finish_kernel, 1, dim3(kNormThreads), st,
                      static_cast<const double*>(partial), parts, max_norm, norm, factor);
}

}  // extern "C"
