// Newton-Schulz orthogonalisation of one matrix per rank:
//   X_0 = G / (|G|_F + 1e-7),  X <- a X + (b A + c A^2) X,  A = X X^T,
// with X [m][n] taken so that m <= n (a tall G is read transposed).
//
// Types.  A step keeps X as the sum of two f16 numbers (22 significand bits)
// and its products run on the f16 matrix instructions with f32 sums.  For f32
// and f16 matrices every factor is such a pair, hi + lo, and a product is
// hi hi + hi lo + lo hi: simulated over Gaussian and fading spectra this is as
// exact as f32 arithmetic (errors of 2e-6 to 6e-6 either way after 5 steps).
// For bf16 matrices a factor is its hi part alone (11 bits, 3 more than the
// result keeps); X itself stays a pair in the a X term, because the early
// steps multiply the small singular directions by about a = 3.4 each and
// would multiply the rounding of X with them (error 1e-2 with X rounded to
// f16 in every step, 2e-4 to 1.7e-3 with the pair; the rounding of the result
// itself is 1.7e-3).
//
// Scale.  Entries of X, A and B = b A + c A^2 are at most about 1, 1.4 and 3;
// they are stored times 2^10, so that the lo parts stay clear of f16's
// smallest steps (2^-24) and values up to 63 fit.
//
// Layout.  X is kept row-major and transposed (both products then read
// k-contiguous rows), A and B are symmetric: only tiles on and below the
// diagonal are computed and each is written twice.
#include "tile.h"
#include "train.h"

namespace emu {

namespace {

constexpr float kScale = 1024.0f, kInvScale = 1.0f / 1024.0f;

template <DType T>
struct Elem;
template <>
struct Elem<DType::F32> { typedef float type; };
template <>
struct Elem<DType::F16> { typedef _Float16 type; };
template <>
struct Elem<DType::BF16> { typedef __bf16 type; };

typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

// v = hi + lo: lo holds what hi's rounding left.
__device__ __forceinline__ void split(float v, _Float16& hi, _Float16& lo) {
  hi = (_Float16)v;
  lo = (_Float16)(v - (float)hi);
}

// |G|^2 of each matrix in parts, in 64 bits (the square of a large f32 has no
// f32 value).  Workgroup (x, y): share x of matrix y.
constexpr int kNormParts = 64;
template <DType T>
__global__ __launch_bounds__(256) void ortho_norm(OrthoArgs a, double* __restrict__ parts) {
  typedef typename Elem<T>::type E;
  const uint64_t count = (uint64_t)a.rows * a.cols;
  const E* in = static_cast<const E*>(a.in[blockIdx.y]);
  double s = 0.0;
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (uint64_t)gridDim.x * 256) {
    const double v = (double)(float)in[i];
    s += v * v;
  }
  for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
  __shared__ double w[4];
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) parts[blockIdx.y * kNormParts + blockIdx.x] = w[0] + w[1] + w[2] + w[3];
}

// One matrix's state.  Pitches are whole 16-byte vectors; what lies past the
// last column is zero.
struct OrthoMat {
  uint64_t x[2], xt[2], a, b;      // byte offsets of the hi part; the lo part follows at + lo_x / lo_a
  uint64_t lo_x, lo_xt, lo_a;
  uint64_t bytes;                  // per matrix
  uint32_t m, n, mp, np;
};

// X_0 = G / (|G| + 1e-7), both layouts.  64 x 64 tiles of X; a tall G is read
// transposed.
template <DType T>
__global__ __launch_bounds__(256) void ortho_load(OrthoArgs a, OrthoMat q, const double* __restrict__ parts,
                                                  char* __restrict__ ws) {
  typedef typename Elem<T>::type E;
  constexpr int B = 64;
  __shared__ float tile[B][B + 1];
  double s = 0.0;
  for (int i = 0; i < kNormParts; ++i) s += parts[blockIdx.z * kNormParts + i];
  // an infinite or NaN entry makes the whole result NaN (the sum of finite
  // squares stays far inside f64's range)
  const double inv = s < (double)INFINITY ? (double)kScale / (sqrt(s) + 1e-7) : (double)NAN;
  const E* in = static_cast<const E*>(a.in[blockIdx.z]);
  char* base = ws + blockIdx.z * q.bytes;
  const uint32_t r0 = blockIdx.y * B, c0 = blockIdx.x * B, x = threadIdx.x % B, y = threadIdx.x / B;   // of G
  for (uint32_t i = y; i < B; i += 4)
    tile[i][x] = r0 + i < a.rows && c0 + x < a.cols
                     ? (float)((double)(float)in[(uint64_t)(r0 + i) * a.cols + c0 + x] * inv)
                     : 0.0f;
  __syncthreads();
  const bool tall = a.rows > a.cols;
  // the layout G has, and the other one
  const uint64_t same = tall ? q.xt[0] : q.x[0], other = tall ? q.x[0] : q.xt[0];
  const uint64_t lo_same = tall ? q.lo_xt : q.lo_x, lo_other = tall ? q.lo_x : q.lo_xt;
  const uint32_t p_same = tall ? q.mp : q.np, p_other = tall ? q.np : q.mp;
  for (uint32_t i = y; i < B; i += 4) {
    _Float16 hi, lo;
    if (r0 + i < a.rows && c0 + x < p_same) {
      split(tile[i][x], hi, lo);
      _Float16* at = reinterpret_cast<_Float16*>(base + same) + (uint64_t)(r0 + i) * p_same + c0 + x;
      at[0] = hi;
      at[lo_same / 2] = lo;
    }
    if (c0 + i < a.cols && r0 + x < p_other) {
      split(tile[x][i], hi, lo);
      _Float16* at = reinterpret_cast<_Float16*>(base + other) + (uint64_t)(c0 + i) * p_other + r0 + x;
      at[0] = hi;
      at[lo_other / 2] = lo;
    }
  }
}

// Tile (i, j), j <= i, of a triangle of tiles, by index.
__device__ __forceinline__ void triangle(uint32_t t, uint32_t& i, uint32_t& j) {
  i = (uint32_t)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
  while (i * (i + 1) / 2 > t) --i;
  while ((i + 1) * (i + 2) / 2 <= t) ++i;
  j = t - i * (i + 1) / 2;
}

// P * Q^T over k: with pairs, hi hi + hi lo + lo hi.
template <class K, bool PAIR>
__device__ __forceinline__ void product(const char* p, uint64_t lo_p, uint32_t rows_p, const char* q, uint64_t lo_q,
                                        uint32_t rows_q, uint32_t pitch, uint32_t lds, typename K::Acc& acc) {
  const uint32_t ld = pitch * 2;
  Operand a{p, ld, (int)rows_p}, b{q, ld, (int)rows_q};
  if constexpr (PAIR) {
    // the small products first
    a.base = p + lo_p;
    K::run(a, b, ld, lds, acc);
    __syncthreads();
    a.base = p;
    b.base = q + lo_q;
    K::run(a, b, ld, lds, acc);
    __syncthreads();
    b.base = q;
  }
  K::run(a, b, ld, lds, acc);
}

// What a symmetric product does with its tile.  kGram: A = X X^T;
// kPoly: B = b A + c A A.
enum SymKind { kGram, kPoly };
template <class K, bool PAIR, SymKind KIND>
__global__ __launch_bounds__(K::threads) void ortho_sym(OrthoMat q, char* ws, uint32_t cur, float cb, float cc) {
  __shared__ __attribute__((aligned(16))) char lds[K::lds_bytes];
  static_assert(K::BM == K::BN, "square tiles");
  uint32_t ti, tj;
  triangle(blockIdx.x, ti, tj);
  char* base = ws + blockIdx.y * q.bytes;
  const uint32_t r0 = ti * K::BM, c0 = tj * K::BN;
  typename K::Acc acc = {};
  const uint32_t pitch = KIND == kGram ? q.np : q.mp;
  const char* src = base + (KIND == kGram ? q.x[cur] : q.a);
  const uint64_t lo = KIND == kGram ? q.lo_x : q.lo_a;
  product<K, PAIR>(src + (uint64_t)r0 * pitch * 2, lo, q.m - r0, src + (uint64_t)c0 * pitch * 2, lo, q.m - c0, pitch,
                   lds_address(lds), acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave / K::WGN, wn = wave % K::WGN;
  _Float16* out = reinterpret_cast<_Float16*>(base + (KIND == kGram ? q.a : q.b));
  const _Float16* am = reinterpret_cast<const _Float16*>(base + q.a);
  const uint64_t lo_a = q.lo_a / 2;
#pragma unroll
  for (int j = 0; j < K::NF; ++j) {
    const uint32_t c = c0 + wn * K::WN + j * 16 + (lane & 15);
#pragma unroll
    for (int i = 0; i < K::MF; ++i) {
      const uint32_t r = r0 + wm * K::WM + i * 16 + 4 * (lane >> 4);
      // row c, columns r .. r + 3 (the upper part), and its mirror
      if (c >= q.m || r >= q.mp) continue;
      const uint64_t at = (uint64_t)c * q.mp + r;
      f16x4 hi, lw;
      f16x4 ahi = {}, alo = {};
      if (KIND == kPoly) {
        ahi = *reinterpret_cast<const f16x4*>(am + at);
        if (PAIR) alo = *reinterpret_cast<const f16x4*>(am + lo_a + at);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = acc[i][j][e] * kInvScale;
        if (KIND == kPoly) v = cb * ((float)ahi[e] + (float)alo[e]) + cc * v;
        if (r + e >= q.m) v = 0.0f;
        _Float16 h, l;
        split(v, h, l);
        hi[e] = h;
        lw[e] = l;
      }
      *reinterpret_cast<f16x4*>(out + at) = hi;
      if (PAIR) *reinterpret_cast<f16x4*>(out + lo_a + at) = lw;
      if (ti != tj) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (r + e < q.m) {
            out[(uint64_t)(r + e) * q.mp + c] = hi[e];
            if (PAIR) out[lo_a + (uint64_t)(r + e) * q.mp + c] = lw[e];
          }
      }
    }
  }
}

// X' = a X + B X into the other buffers, or, in the last step, into the
// output.  First operand B (rows i), second X transposed (rows k).
template <DType T, class K, bool PAIR, bool LAST>
__global__ __launch_bounds__(K::threads) void ortho_step(OrthoArgs a, OrthoMat q, char* ws, uint32_t cur, float ca,
                                                         uint32_t tm, uint32_t tn) {
  typedef typename Elem<T>::type E;
  __shared__ __attribute__((aligned(16))) char lds[K::lds_bytes];
  uint32_t m, n;
  tile_of(blockIdx.x, tm, tn, 8, m, n);
  char* base = ws + blockIdx.y * q.bytes;
  const uint32_t r0 = m * K::BM, c0 = n * K::BN;
  typename K::Acc acc = {};
  product<K, PAIR>(base + q.b + (uint64_t)r0 * q.mp * 2, q.lo_a, q.m - r0,
                   base + q.xt[cur] + (uint64_t)c0 * q.mp * 2, q.lo_xt, q.n - c0, q.mp, lds_address(lds), acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave / K::WGN, wn = wave % K::WGN;
  const _Float16* xt = reinterpret_cast<const _Float16*>(base + q.xt[cur]);
  _Float16* nxt = reinterpret_cast<_Float16*>(base + q.xt[cur ^ 1]);
  _Float16* nx = reinterpret_cast<_Float16*>(base + q.x[cur ^ 1]);
  E* out = static_cast<E*>(a.out[blockIdx.y]);
  const bool tall = a.rows > a.cols;
#pragma unroll
  for (int j = 0; j < K::NF; ++j) {
    const uint32_t k = c0 + wn * K::WN + j * 16 + (lane & 15);
#pragma unroll
    for (int i = 0; i < K::MF; ++i) {
      const uint32_t r = r0 + wm * K::WM + i * 16 + 4 * (lane >> 4);
      if (r >= q.mp || k >= q.np) continue;
      f16x4 xh = {}, xl = {};
      if (k < q.n) {
        xh = *reinterpret_cast<const f16x4*>(xt + (uint64_t)k * q.mp + r);
        xl = *reinterpret_cast<const f16x4*>(xt + q.lo_xt / 2 + (uint64_t)k * q.mp + r);
      }
      f16x4 hi, lw;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = ca * ((float)xh[e] + (float)xl[e]) + acc[i][j][e] * kInvScale;
        if (r + e >= q.m || k >= q.n) v[e] = 0.0f;
        _Float16 h, l;
        split(v[e], h, l);
        hi[e] = h;
        lw[e] = l;
      }
      if constexpr (LAST) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (r + e < q.m && k < q.n)
            out[tall ? (uint64_t)k * a.cols + r + e : (uint64_t)(r + e) * a.cols + k] = (E)(v[e] * kInvScale);
      } else {
        if (k < q.n) {
          *reinterpret_cast<f16x4*>(nxt + (uint64_t)k * q.mp + r) = hi;
          *reinterpret_cast<f16x4*>(nxt + q.lo_xt / 2 + (uint64_t)k * q.mp + r) = lw;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (r + e < q.m) {
            nx[(uint64_t)(r + e) * q.np + k] = hi[e];
            if (PAIR) nx[q.lo_x / 2 + (uint64_t)(r + e) * q.np + k] = lw[e];
          }
      }
    }
  }
}

typedef TileMma<DType::F16, 256, 256, 2, 4> Big;
typedef TileMma<DType::F16, 128, 128, 2, 2> Mid;

OrthoMat layout(const OrthoArgs& a) {
  OrthoMat q{};
  q.m = std::min(a.rows, a.cols);
  q.n = std::max(a.rows, a.cols);
  q.mp = (uint32_t)align_up(q.m, 8);
  q.np = (uint32_t)align_up(q.n, 8);
  size_t at = 0;
  auto take = [&](size_t n) { const size_t p = at; at = align_up(at + n, 256); return p; };
  const size_t x = (size_t)q.m * q.np * 2, xt = (size_t)q.n * q.mp * 2, s = (size_t)q.m * q.mp * 2;
  q.lo_x = align_up(x, 256);
  q.lo_xt = align_up(xt, 256);
  q.lo_a = align_up(s, 256);
  for (int i = 0; i < 2; ++i) {
    q.x[i] = take(2 * q.lo_x);
    q.xt[i] = take(2 * q.lo_xt);
  }
  q.a = take(2 * q.lo_a);
  q.b = take(2 * q.lo_a);
  q.bytes = at;
  return q;
}

uint32_t ceil_div(uint32_t a, uint32_t b) { return (a + b - 1) / b; }

template <class K, bool PAIR, SymKind KIND>
void launch_sym(const OrthoMat& q, uint32_t nmat, char* ws, uint32_t cur, float cb, float cc, hipStream_t s) {
  const uint32_t t = ceil_div(q.m, K::BM);
  hipLaunchKernelGGL((ortho_sym<K, PAIR, KIND>), dim3(t * (t + 1) / 2, nmat), dim3(K::threads), 0, s, q, ws, cur, cb, cc);
}
template <DType T, class K, bool PAIR>
void launch_step(const OrthoArgs& a, const OrthoMat& q, char* ws, uint32_t cur, float ca, bool last, hipStream_t s) {
  const uint32_t tm = ceil_div(q.m, K::BM), tn = ceil_div(q.n, K::BN);
  if (last)
    hipLaunchKernelGGL((ortho_step<T, K, PAIR, true>), dim3(tm * tn, a.nranks), dim3(K::threads), 0, s, a, q, ws, cur,
                       ca, tm, tn);
  else
    hipLaunchKernelGGL((ortho_step<T, K, PAIR, false>), dim3(tm * tn, a.nranks), dim3(K::threads), 0, s, a, q, ws, cur,
                       ca, tm, tn);
}

template <DType T>
hipError_t run(const OrthoArgs& a, char* workspace, hipStream_t s) {
  constexpr bool PAIR = T != DType::BF16;
  const OrthoMat q = layout(a);
  double* parts = reinterpret_cast<double*>(workspace);
  char* ws = workspace + align_up((size_t)a.nranks * kNormParts * sizeof(double), 256);
  hipLaunchKernelGGL(ortho_norm<T>, dim3(kNormParts, a.nranks), dim3(256), 0, s, a, parts);
  hipLaunchKernelGGL(ortho_load<T>, dim3(ceil_div(a.cols, 64), ceil_div(a.rows, 64), a.nranks), dim3(256), 0, s, a, q,
                     parts, ws);
  const uint64_t t = ceil_div(q.m, 256);
  const bool sym_big = t * (t + 1) / 2 * a.nranks >= (uint64_t)a.cus;
  const bool step_big = t * ceil_div(q.n, 256) * a.nranks >= (uint64_t)a.cus;
  uint32_t cur = 0;
  for (int i = 0; i < a.steps; ++i, cur ^= 1) {
    const float* c = a.coeffs + 3 * i;
    if (sym_big) {
      launch_sym<Big, PAIR, kGram>(q, a.nranks, ws, cur, 0.0f, 0.0f, s);
      launch_sym<Big, PAIR, kPoly>(q, a.nranks, ws, cur, c[1], c[2], s);
    } else {
      launch_sym<Mid, PAIR, kGram>(q, a.nranks, ws, cur, 0.0f, 0.0f, s);
      launch_sym<Mid, PAIR, kPoly>(q, a.nranks, ws, cur, c[1], c[2], s);
    }
    if (step_big) launch_step<T, Big, PAIR>(a, q, ws, cur, c[0], i + 1 == a.steps, s);
    else launch_step<T, Mid, PAIR>(a, q, ws, cur, c[0], i + 1 == a.steps, s);
  }
  return hipGetLastError();
}

}  // namespace

size_t ortho_space(const OrthoArgs& a) {
  return align_up((size_t)a.nranks * kNormParts * sizeof(double), 256) + (size_t)a.nranks * layout(a).bytes;
}

int orthogonalize(const OrthoArgs& a, char* workspace, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (a.type) {
    case DType::F32: return run<DType::F32>(a, workspace, s);
    case DType::F16: return run<DType::F16>(a, workspace, s);
    default: return run<DType::BF16>(a, workspace, s);
  }
}

}  // namespace emu
