// Load-balance loss of a mixture-of-experts router over every rank's tokens:
//   p_t = softmax(z_t),  f_e = count_e / (N k),  P_e = (1/N) sum_t p_te,
//   L = coef E sum_e f_e P_e,
//   dL/dz_te = coef (E/N) p_te (f_e - sum_e' f_e' p_te'),
// N the counted tokens of all ranks (those with at least one chosen expert).
//
// Three launches.  balance_rows reads every logit once: a group of lanes
// holds a row in registers, adds its probabilities to the group's own column
// sums and its choices to the workgroup's integer counts, and leaves one row
// of partial sums per workgroup.  balance_join adds those rows in ascending
// order (so results repeat bit for bit) in 64 bits and forms f.
// balance_grad reads the logits again and writes their gradients.
#include "device_ops.h"
#include "train.h"

namespace emu {

namespace {

constexpr int kBalThreads = 256;
constexpr int kBalWaves = kBalThreads / 64;

template <DType T>
struct Elem;
template <>
struct Elem<DType::F32> { typedef float type; };
template <>
struct Elem<DType::F16> { typedef _Float16 type; };
template <>
struct Elem<DType::BF16> { typedef __bf16 type; };

// One row in a group's registers: lane `l` of `group` lanes holds columns
// (l + i * group) * VEC + v.  Columns past the row read as -inf.
template <DType T, int VEC, int NI>
struct Row {
  using E = typename Elem<T>::type;
  typedef E EV __attribute__((ext_vector_type(VEC)));
  float z[NI][VEC];
  __device__ __forceinline__ void load(const void* logits, uint64_t row, uint32_t nexperts, uint32_t l, uint32_t group) {
    const E* p = static_cast<const E*>(logits) + row * nexperts;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint32_t c = (l + i * group) * VEC;
      if (c < nexperts) {
        if constexpr (VEC == 1) {
          z[i][0] = (float)p[c];
        } else {
          const EV x = *reinterpret_cast<const EV*>(p + c);
#pragma unroll
          for (int v = 0; v < VEC; ++v) z[i][v] = (float)x[v];
        }
      } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) z[i][v] = -INFINITY;
      }
    }
  }
  __device__ __forceinline__ void store(void* out, uint64_t row, uint32_t nexperts, uint32_t l, uint32_t group) const {
    E* p = static_cast<E*>(out) + row * nexperts;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint32_t c = (l + i * group) * VEC;
      if (c < nexperts) {
        if constexpr (VEC == 1) {
          p[c] = (E)z[i][0];
        } else {
          EV x;
#pragma unroll
          for (int v = 0; v < VEC; ++v) x[v] = (E)z[i][v];
          *reinterpret_cast<EV*>(p + c) = x;
        }
      }
    }
  }
  // z -> softmax(z).  A row whose logits are all -inf has no probabilities
  // and becomes zeros.
  __device__ __forceinline__ void softmax(uint32_t group) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v) m = fmaxf(m, z[i][v]);
    for (uint32_t d = 1; d < group; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    if (m == -INFINITY) m = 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        z[i][v] = __builtin_amdgcn_exp2f((z[i][v] - m) * 1.44269504088896341f);
        s += z[i][v];
      }
    for (uint32_t d = 1; d < group; d <<= 1) s += __shfl_xor(s, d);
    const float r = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v) z[i][v] *= r;
  }
};

// Whether token `row` chose any expert, seen by every lane of its group; adds
// its choices to `counts` (LDS) if given.
__device__ __forceinline__ bool chosen(const int32_t* experts, uint64_t row, uint32_t topk, uint32_t nexperts,
                                       uint32_t l, uint32_t group, uint32_t* counts) {
  int any = 0;
  for (uint32_t k = l; k < topk; k += group) {
    const uint32_t e = (uint32_t)experts[row * topk + k];
    if (e < nexperts) {
      any = 1;
      if (counts) atomicAdd(&counts[e], 1u);
    }
  }
  for (uint32_t d = 1; d < group; d <<= 1) any |= __shfl_xor(any, d);
  return any != 0;
}

// Which rank and rows workgroup `b` has: rank r's tokens are split into
// blocks of `rows` tokens.
struct BalanceGrid {
  uint32_t block0[kMaxRanks + 1];
  uint32_t rows;
};
__device__ __forceinline__ uint32_t rank_of(const BalanceGrid& g, uint32_t nranks, uint32_t b) {
  uint32_t r = 0;
  while (r + 1 < nranks && b >= g.block0[r + 1]) ++r;
  return r;
}

template <DType T, int VEC, int NI>
__global__ __launch_bounds__(kBalThreads) void balance_rows(BalanceArgs a, BalanceGrid g, uint32_t group,
                                                          float* __restrict__ psum, uint32_t* __restrict__ pcount,
                                                          uint32_t* __restrict__ pvalid) {
  extern __shared__ char lds[];
  float* sums = reinterpret_cast<float*>(lds);                     // [kBalWaves][nexperts]
  uint32_t* counts = reinterpret_cast<uint32_t*>(sums + kBalWaves * a.nexperts);
  __shared__ uint32_t nvalid;
  const uint32_t b = blockIdx.x, r = rank_of(g, a.nranks, b);
  const uint32_t begin = (b - g.block0[r]) * g.rows, end = min(begin + g.rows, a.tokens[r]);
  const uint32_t l = threadIdx.x & (group - 1), slot = threadIdx.x / group, slots = kBalThreads / group;
  for (uint32_t e = threadIdx.x; e < a.nexperts; e += kBalThreads) counts[e] = 0;
  if (threadIdx.x == 0) nvalid = 0;
  __syncthreads();
  float acc[NI][VEC] = {};
  uint32_t mine = 0;
  for (uint32_t first = begin; first < end; first += slots) {
    const uint32_t row = first + slot;
    if (row >= end) continue;                                      // whole groups
    if (!chosen(a.experts[r], row, a.topk, a.nexperts, l, group, counts)) continue;
    Row<T, VEC, NI> z;
    z.load(a.logits[r], row, a.nexperts, l, group);
    z.softmax(group);
    if (l == 0) ++mine;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v) acc[i][v] += z.z[i][v];
  }
  if (mine) atomicAdd(&nvalid, mine);
  // the groups of a wave hold the same columns: add them, then the waves
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      float s = acc[i][v];
      for (uint32_t d = group; d < 64; d <<= 1) s += __shfl_xor(s, d);
      const uint32_t c = (l + i * group) * VEC + v;
      if ((threadIdx.x & 63) < group && c < a.nexperts) sums[(threadIdx.x >> 6) * a.nexperts + c] = s;
    }
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < a.nexperts; e += kBalThreads) {
    float s = 0.0f;
    for (int w = 0; w < kBalWaves; ++w) s += sums[w * a.nexperts + e];
    psum[(uint64_t)b * a.nexperts + e] = s;
    pcount[(uint64_t)b * a.nexperts + e] = counts[e];
  }
  if (threadIdx.x == 0) pvalid[b] = nvalid;
}

// One workgroup per 16 experts, 16 lanes each: lane k of an expert adds the
// partial rows k, k + 16, ... of a rank, and the 16 parts are added in order.
constexpr int kJoinExperts = 16, kJoinLanes = 16;
__global__ __launch_bounds__(kJoinExperts* kJoinLanes) void balance_join(BalanceArgs a, BalanceGrid g,
                                                                         const float* __restrict__ psum,
                                                                         const uint32_t* __restrict__ pcount,
                                                                         const uint32_t* __restrict__ pvalid,
                                                                         float* __restrict__ f,
                                                                         double* __restrict__ term,
                                                                         float* __restrict__ inv) {
  __shared__ double dsum[kJoinLanes][kJoinExperts];
  __shared__ unsigned long long csum[kJoinLanes][kJoinExperts];
  const uint32_t le = threadIdx.x % kJoinExperts, k = threadIdx.x / kJoinExperts;
  const uint32_t e = blockIdx.x * kJoinExperts + le;
  const uint32_t nblocks = g.block0[a.nranks];
  unsigned long long n = 0;
  for (uint32_t b = threadIdx.x; b < nblocks; b += kJoinExperts * kJoinLanes) n += pvalid[b];
  csum[k][le] = n;
  __syncthreads();
  n = 0;
  for (int i = 0; i < kJoinLanes; ++i)
    for (int j = 0; j < kJoinExperts; ++j) n += csum[i][j];
  double s = 0.0;
  unsigned long long total = 0;
  for (uint32_t r = 0; r < a.nranks; ++r) {
    unsigned long long c = 0;
    if (e < a.nexperts)
      for (uint32_t b = g.block0[r] + k; b < g.block0[r + 1]; b += kJoinLanes) {
        s += (double)psum[(uint64_t)b * a.nexperts + e];
        c += pcount[(uint64_t)b * a.nexperts + e];
      }
    __syncthreads();
    csum[k][le] = c;
    __syncthreads();
    if (k == 0 && e < a.nexperts) {
      c = 0;
      for (int i = 0; i < kJoinLanes; ++i) c += csum[i][le];
      a.counts[(uint64_t)r * a.nexperts + e] = (int64_t)c;
      total += c;
    }
  }
  dsum[k][le] = s;
  __syncthreads();
  if (k == 0 && e < a.nexperts) {
    s = 0.0;
    for (int i = 0; i < kJoinLanes; ++i) s += dsum[i][le];
    a.counts[(uint64_t)a.nranks * a.nexperts + e] = (int64_t)total;
    const double share = n ? (double)total / ((double)n * a.topk) : 0.0;
    f[e] = (float)share;
    term[e] = n ? share * (s / (double)n) : 0.0;
    if (e == 0) *inv = n ? (float)((double)a.coef * a.nexperts / (double)n) : 0.0f;
  }
}

template <DType T, int VEC, int NI>
__global__ __launch_bounds__(kBalThreads) void balance_grad(BalanceArgs a, BalanceGrid g, uint32_t group,
                                                          const float* __restrict__ f, const float* __restrict__ inv) {
  const uint32_t b = blockIdx.x, r = rank_of(g, a.nranks, b);
  const uint32_t begin = (b - g.block0[r]) * g.rows, end = min(begin + g.rows, a.tokens[r]);
  const uint32_t l = threadIdx.x & (group - 1), slot = threadIdx.x / group, slots = kBalThreads / group;
  const float scale = *inv;
  float fe[NI][VEC];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const uint32_t c = (l + i * group) * VEC + v;
      fe[i][v] = c < a.nexperts ? f[c] : 0.0f;
    }
  for (uint32_t first = begin; first < end; first += slots) {
    const uint32_t row = first + slot;
    if (row >= end) continue;
    Row<T, VEC, NI> z;
    if (chosen(a.experts[r], row, a.topk, a.nexperts, l, group, nullptr)) {
      z.load(a.logits[r], row, a.nexperts, l, group);
      z.softmax(group);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int v = 0; v < VEC; ++v) dot += fe[i][v] * z.z[i][v];
      for (uint32_t d = 1; d < group; d <<= 1) dot += __shfl_xor(dot, d);
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int v = 0; v < VEC; ++v) z.z[i][v] = scale * z.z[i][v] * (fe[i][v] - dot);
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int v = 0; v < VEC; ++v) z.z[i][v] = 0.0f;
    }
    z.store(a.dlogits[r], row, a.nexperts, l, group);
  }
}

__global__ __launch_bounds__(64) void balance_total(BalanceArgs a, const double* __restrict__ term) {
  double s = 0.0;
  for (uint32_t e = threadIdx.x; e < a.nexperts; e += 64) s += term[e];
  for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
  if (threadIdx.x == 0) *a.loss = (float)((double)a.coef * a.nexperts * s);
}

// Tokens per workgroup: 32 rows in flight at least, more when that still
// leaves four workgroups per CU.
BalanceGrid balance_grid(const BalanceArgs& a) {
  uint64_t all = 0;
  for (uint32_t r = 0; r < a.nranks; ++r) all += a.tokens[r];
  BalanceGrid g{};
  const uint64_t want = (all + 4u * a.cus - 1) / (4u * a.cus);
  g.rows = 32;
  while (g.rows < want && g.rows < 4096) g.rows *= 2;
  for (uint32_t r = 0; r < a.nranks; ++r) g.block0[r + 1] = g.block0[r] + (a.tokens[r] + g.rows - 1) / g.rows;
  return g;
}

struct BalanceSpace {
  size_t psum, pcount, pvalid, f, term, inv, bytes;
};
BalanceSpace layout(const BalanceArgs& a, uint32_t nblocks) {
  BalanceSpace s{};
  size_t at = 0;
  auto take = [&](size_t n) { const size_t p = at; at = align_up(at + n, 256); return p; };
  s.psum = take((size_t)nblocks * a.nexperts * 4);
  s.pcount = take((size_t)nblocks * a.nexperts * 4);
  s.pvalid = take((size_t)nblocks * 4);
  s.f = take((size_t)a.nexperts * 4);
  s.term = take((size_t)a.nexperts * 8);
  s.inv = take(4);
  s.bytes = at;
  return s;
}

template <DType T, int VEC, int NI>
hipError_t launch(const BalanceArgs& a, const BalanceGrid& g, uint32_t group, char* ws, hipStream_t s) {
  const uint32_t nblocks = g.block0[a.nranks];
  const BalanceSpace m = layout(a, nblocks);
  float* psum = reinterpret_cast<float*>(ws + m.psum);
  uint32_t* pcount = reinterpret_cast<uint32_t*>(ws + m.pcount);
  uint32_t* pvalid = reinterpret_cast<uint32_t*>(ws + m.pvalid);
  float* f = reinterpret_cast<float*>(ws + m.f);
  double* term = reinterpret_cast<double*>(ws + m.term);
  float* inv = reinterpret_cast<float*>(ws + m.inv);
  if (nblocks)
    hipLaunchKernelGGL((balance_rows<T, VEC, NI>), dim3(nblocks), dim3(kBalThreads),
                       (kBalWaves + 1) * a.nexperts * 4, s, a, g, group, psum, pcount, pvalid);
  hipLaunchKernelGGL(balance_join, dim3((a.nexperts + kJoinExperts - 1) / kJoinExperts),
                     dim3(kJoinExperts * kJoinLanes), 0, s, a, g, psum, pcount, pvalid, f, term, inv);
  hipLaunchKernelGGL(balance_total, dim3(1), dim3(64), 0, s, a, term);
  if (nblocks && a.grad)
    hipLaunchKernelGGL((balance_grad<T, VEC, NI>), dim3(nblocks), dim3(kBalThreads), 0, s, a, g, group, f, inv);
  return hipGetLastError();
}

template <DType T>
hipError_t dispatch(const BalanceArgs& a, char* ws, hipStream_t s) {
  constexpr int V = Unit<T>::elems;
  const BalanceGrid g = balance_grid(a);
  const bool whole = a.nexperts % V == 0;      // every row starts on a vector
  const uint32_t units = whole ? a.nexperts / V : a.nexperts;
  uint32_t group = 1;
  while (group < 64 && group < units) group *= 2;
  const uint32_t ni = (units + group - 1) / group;
  if (whole) {
    if (ni == 1) return launch<T, V, 1>(a, g, group, ws, s);
    if (ni == 2) return launch<T, V, 2>(a, g, group, ws, s);
    return launch<T, V, 4>(a, g, group, ws, s);
  }
  if (ni == 1) return launch<T, 1, 1>(a, g, group, ws, s);
  if (ni <= 4) return launch<T, 1, 4>(a, g, group, ws, s);
  return launch<T, 1, 16>(a, g, group, ws, s);
}

}  // namespace

size_t balance_space(const BalanceArgs& a) { return layout(a, balance_grid(a).block0[a.nranks]).bytes; }

int balance_loss(const BalanceArgs& a, char* workspace, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (a.type) {
    case DType::F32: return dispatch<DType::F32>(a, workspace, s);
    case DType::F16: return dispatch<DType::F16>(a, workspace, s);
    default: return dispatch<DType::BF16>(a, workspace, s);
  }
}

}  // namespace emu
