// Residual addition with root-mean-square norm, forward and backward (gfx950):
// what a transformer block runs on the token rows before the expert layer.
//
//   h = x + res (rounded to the storage type),  rs = 1 / sqrt(mean(h^2) + eps),
//   y = h * rs * w,  and optionally the MXFP8 copy of y along each row.
//   n = h * rs,  g = dy * w:  dx = dh + rs * (g - n * mean(g * n)),  dw = sum_t dy * n
//
// Memory-bound in both directions: every element is read and written once, and
// a whole row stays in the registers of the 1 to 12 waves that share it, so
// the norm and the quantisation cost no second pass. 16384 x 2048 bf16 with a
// residual: forward 42.7 us (6.3 TB/s; a plain copy reaches 5.1), 51 to 57
// with the MXFP8 copy, in binary32 92 us (5.8 TB/s), backward 48.3 us with dw; one
// token 3.0 us, 2.7 of them a launch's own. See include/moe.h for the contract of each entry point.
#include "mx_common.h"

#include <type_traits>

namespace moe {

namespace {

// A row lies in the registers of W waves, U 16-byte pieces a lane. The smallest
// of these that holds the row (16 waves of one workgroup would leave the
// backward kernel 128 registers each, fewer than it needs, so 12 is the most):
// pieces past the row are loaded and not used, so a tighter fit is faster
// (4096 x 4096 bf16 backward: 35 us with W = 4, 33 with W = 2).
template <typename T> constexpr int kNormMaxWaves = MOE_MAX_NORM_D / (64 * 4 * kVec<T>);   // 6 (bf16), 12 (binary32)

template <typename T, class F> void norm_shape(int d, F&& launch) {
  const int per = 64 * kVec<T>;   // values a wave holds in one piece a lane
  using std::integral_constant;
  if (d <= 2 * per) launch(integral_constant<int, 1>(), integral_constant<int, 2>());
  else if (d <= 4 * per) launch(integral_constant<int, 1>(), integral_constant<int, 4>());
  else if (d <= 8 * per) launch(integral_constant<int, 2>(), integral_constant<int, 4>());
  else if (d <= 16 * per) launch(integral_constant<int, 4>(), integral_constant<int, 4>());
  else launch(integral_constant<int, kNormMaxWaves<T>>(), integral_constant<int, 4>());
}

struct NormArgs {
  const void* x;
  const void* res;   // null: h = x, not written
  const void* w;
  void* h;
  void* y;           // null: only the MXFP8 copy
  uint8_t* q;        // null: no MXFP8 copy
  uint8_t* s;
  float* rstd;       // null: not wanted
  int T, d;
  float eps;
};

// Piece c of a row: a wave-uniform base and a 32-bit byte offset, so that the
// address costs one register.
template <bool NT, typename T> MOE_DEV V16 load_piece(const T* row, uint32_t c) {
  return load16<NT>(reinterpret_cast<const char*>(row) + c * 16u);
}
template <bool NT, typename T> MOE_DEV void store_piece(T* row, uint32_t c, const V16& v) {
  store16<NT>(reinterpret_cast<char*>(row) + c * 16u, v);
}
MOE_DEV uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }

// Sum of a lane's V values as a tree, which keeps the roundings of a row's sum
// few in a row: its error is every element's of its row.
template <int V> MOE_DEV float tree_sum(const float (&v)[V]) {
  float s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = v[i];
#pragma unroll
  for (int o = V / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) s[i] += s[i + o];
  return s[0];
}

// Sum over the W waves of a row; `red` holds one sum per wave of the
// workgroup and is not reused before another barrier.
template <int W, typename S> MOE_DEV S row_sum(S v, S* red, int wave) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if constexpr (W == 1) return v;
  if ((threadIdx.x & 63) == 0) red[wave] = v;
  __syncthreads();
  S t = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) t += red[i];
  return t;
}

template <int W> constexpr int kNormThreads = W == 1 ? 256 : 64 * W;   // four rows, or one

// NT (launches that stream): x and res are read for the last time, h is next
// read by the backward pass; y is read at once and goes through the caches.
// Norm, router and permute of 16384 x 2048 rows: 137 us without, 112 us so,
// 128 us with y past the caches too.
template <typename T, int W, int U, bool MX, bool NT>
__global__ void __launch_bounds__(kNormThreads<W>) add_rmsnorm_kernel(NormArgs a) {
  constexpr int V = kVec<T>;
  __shared__ double red[W];
  __shared__ uint32_t words[MX && W == 1 ? 4 * U : 1][4];   // scale words of four rows
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // a wave past the last row works on it again and stores nothing
  const size_t t1 = W == 1 ? (size_t)blockIdx.x * 4 + wave : blockIdx.x, t = t1 < (size_t)a.T ? t1 : a.T - 1;
  const int d = a.d;
  const uint32_t nvec = d / V, nst = t1 == t ? nvec : 0, c0 = (W == 1 ? 0 : wave * 64) + lane;
  // all loads first, unconditional: a piece past the row reads its last one
  const T* xp = static_cast<const T*>(a.x) + t * d;
  const T* rp = static_cast<const T*>(a.res ? a.res : a.x) + t * d;
  const T* wp = static_cast<const T*>(a.w);
  V16 hv[U], rv[U], wv[U];
#pragma unroll
  for (int u = 0; u < U; ++u) hv[u] = load_piece<NT>(xp, umin(c0 + 64 * W * u, nvec - 1));
  if (a.res) {
#pragma unroll
    for (int u = 0; u < U; ++u) rv[u] = load_piece<NT>(rp, umin(c0 + 64 * W * u, nvec - 1));
  }
#pragma unroll
  for (int u = 0; u < U; ++u) wv[u] = load_piece<false>(wp, umin(c0 + 64 * W * u, nvec - 1));
  double sum = 0;   // of squares
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool in = c0 + 64 * W * u < nvec;
    float f[V];
    unpack(hv[u], f);
    if (a.res) {
      float r[V];
      unpack(rv[u], r);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] += r[i];
      hv[u] = pack(f);     // the norm is taken of h as it is stored
      unpack(hv[u], f);
      if (c0 + 64 * W * u < nst) store_piece<NT>(static_cast<T*>(a.h) + t * d, c0 + 64 * W * u, hv[u]);
    }
    // every square and every sum in 64 bits (16384 x 2048 43.3 us, with groups of
    // eight squares added in binary32 43.1): a square of 2e19 is infinite there
    double sq = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) sq = fma(static_cast<double>(f[i]), static_cast<double>(f[i]), sq);
    sum += in ? sq : 0.0;
  }
  sum = row_sum<W>(sum, red, wave);
  const double rs = 1.0 / sqrt(sum / d + a.eps);
  if (a.rstd && c0 < min(nst, 1u)) a.rstd[t] = static_cast<float>(rs);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t c = c0 + 64 * W * u;
    float f[V], w[V];
    unpack(hv[u], f);
    unpack(wv[u], w);
    // the product in 64 bits: y is rounded to binary32 once, and no factor of it
    // leaves the range that y itself does not leave (all of 33 M bf16 values are
    // the exact ones rounded by way of binary32). Binary32 products with the root
    // in two terms, which do leave it, take 43.0 us where this takes 42.5 to 43.0
    // (16384 x 2048 with a residual), 55.3 for 55.8 with the MXFP8 copy, 46.6 for
    // 48.4 without a residual (32768 x 2048), 8.2 for 8.5 at 2048 rows
#pragma unroll
    for (int i = 0; i < V; ++i)
      f[i] = static_cast<float>(static_cast<double>(f[i]) * rs * static_cast<double>(w[i]));
    const V16 yv = pack(f);
    if (a.y && c < nst) store_piece<false>(static_cast<T*>(a.y) + t * d, c, yv);
    if constexpr (MX) {
      // four lanes hold a block of 32 values, sixteen the four blocks of a
      // scale word (nvec is a multiple of 16: no group straddles the row's end)
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = mag_max2(m, yv.w[i]);
      m = max2(m, __shfl_xor(m, 1, 64));
      m = max2(m, __shfl_xor(m, 2, 64));
      const BlockScale bs = block_scale(max_half(m));
      const uint2 o = make_uint2(encode_quad(yv.w[0], yv.w[1], bs), encode_quad(yv.w[2], yv.w[3], bs));
      const uint32_t code = static_cast<uint32_t>(bs.x + 127);
      const uint32_t word = code | __shfl_down(code, 4, 64) << 8 | __shfl_down(code, 8, 64) << 16 |
                            __shfl_down(code, 12, 64) << 24;
      if (c < nst) {
        reinterpret_cast<uint2*>(a.q + t * d)[c] = o;
        if constexpr (W > 1) {
          if ((lane & 15) == 0)
            *reinterpret_cast<uint32_t*>(a.s + 4 * (static_cast<size_t>(a.T) * (c >> 4) + t)) = word;
        }
      }
      if constexpr (W == 1) {
        if ((lane & 15) == 0) words[4 * u + (lane >> 4)][wave] = word;
      }
    }
  }
  if constexpr (MX && W == 1) {
    // the four rows' words of a column group are neighbours: one store of
    // 16-byte runs for all of them (52.8 us with a store a word, 50.9 so)
    __syncthreads();
    const uint32_t c = threadIdx.x >> 2;
    const size_t row = (size_t)blockIdx.x * 4 + (threadIdx.x & 3);
    if (c < nvec / 16 && row < (size_t)a.T)
      *reinterpret_cast<uint32_t*>(a.s + 4 * (static_cast<size_t>(a.T) * c + row)) = words[c][threadIdx.x & 3];
  }
}


// ------------------------------------------------------------------ backward
struct NormBwdArgs {
  const void* dy;
  const void* h;
  const void* w;
  const float* rstd;
  const void* dh;    // null: nothing arrives along the residual
  void* dx;
  float* part;       // [gridDim.x][d] sums of dy * n over a workgroup's rows; null: dw is not wanted
  int T, d;
};

// Workgroups stride over the rows and keep their share of dw in registers
// (44 us of the 48.3; the rest adds the parts). Loads of the next row under
// the current one's work were slower (49.8 us): the other waves cover them.
template <typename T, int W, int U, bool NT>
__global__ void __launch_bounds__(kNormThreads<W>) rmsnorm_bwd_kernel(NormBwdArgs a) {
  constexpr int V = kVec<T>, RPB = W == 1 ? 4 : 1;
  __shared__ float red[2][W > 4 ? W : 4];
  __shared__ float sums[W == 1 ? 64 * U * V : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int d = a.d;
  const uint32_t nvec = d / V, c0 = (W == 1 ? 0 : wave * 64) + lane;
  const T* wp = static_cast<const T*>(a.w);
  V16 wv[U];
  float dw[U][V];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    wv[u] = load_piece<false>(wp, umin(c0 + 64 * W * u, nvec - 1));
#pragma unroll
    for (int i = 0; i < V; ++i) dw[u][i] = 0.f;
  }
  int par = 0;
  for (size_t t = (size_t)blockIdx.x * RPB + (W == 1 ? wave : 0); t < (size_t)a.T; t += (size_t)gridDim.x * RPB) {
    const T* gp = static_cast<const T*>(a.dy) + t * d;
    const T* hp = static_cast<const T*>(a.h) + t * d;
    const T* rp = static_cast<const T*>(a.dh ? a.dh : a.dy) + t * d;
    V16 gv[U], hv[U], rv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      gv[u] = load_piece<NT>(gp, umin(c0 + 64 * W * u, nvec - 1));
      hv[u] = load_piece<NT>(hp, umin(c0 + 64 * W * u, nvec - 1));
    }
    if (a.dh) {
#pragma unroll
      for (int u = 0; u < U; ++u) rv[u] = load_piece<NT>(rp, umin(c0 + 64 * W * u, nvec - 1));
    }
    const float rs = a.rstd[t];
    float part[U];     // sums of g * n
    // held packed across the phases: unpacked copies would take 150 registers
#pragma unroll
    for (int u = 0; u < U; ++u) pin(wv[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = c0 + 64 * W * u < nvec;
      float g[V], n[V], w[V];
      unpack(gv[u], g);
      unpack(hv[u], n);
      unpack(wv[u], w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float p = in ? g[i] * (n[i] * rs) : 0.f;
        dw[u][i] += p;
        g[i] = p * w[i];
      }
      part[u] = tree_sum(g);
    }
    const float dot = row_sum<W>(tree_sum(part), red[par], wave);
    par ^= 1;          // the next row's sums must not overwrite these before every wave has read them
    const float mean = dot / (float)d;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      pin(gv[u]);
      pin(hv[u]);
      pin(wv[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t c = c0 + 64 * W * u;
      float g[V], n[V], w[V], r[V];
      unpack(gv[u], g);
      unpack(hv[u], n);
      unpack(wv[u], w);
      if (a.dh) unpack(rv[u], r);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float v = rs * (g[i] * w[i] - (n[i] * rs) * mean);
        g[i] = a.dh ? r[i] + v : v;
      }
      if (c < nvec) store_piece<false>(static_cast<T*>(a.dx) + t * d, c, pack(g));
    }
  }
  if (!a.part) return;
  float* out = a.part + (size_t)blockIdx.x * d;
  if constexpr (W == 1) {
    // the four waves' sums, added in wave order
    for (int k = 0; k < 4; ++k) {
      if (wave == k) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float* p = sums + (64 * u + lane) * V + i;
            *p = k ? *p + dw[u][i] : dw[u][i];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < d; c += 256) out[c] = sums[c];
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t c = c0 + 64 * W * u;
      if (c < nvec) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
          *reinterpret_cast<float4*>(out + (size_t)c * V + i) = make_float4(dw[u][i], dw[u][i + 1], dw[u][i + 2], dw[u][i + 3]);
      }
    }
  }
}

// dw[c] = sum over the parts, in a fixed order: 128 threads of a workgroup take
// every 128th part of 4 columns each, four loads in flight, then their sums
// are added in LDS. 32 columns a workgroup: 1024 parts of 2048 columns take
// 3 us less than with 64.
constexpr int kRedCols = 32, kRedRows = 1024 / (kRedCols / 4);
template <typename T>
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* __restrict__ part, int parts, int d,
                                                       T* __restrict__ dw) {
  constexpr int CL = kRedCols / 4, UN = 4;
  __shared__ float4 acc[kRedRows][CL];
  const int ci = threadIdx.x % CL, gi = threadIdx.x / CL;
  const int c = blockIdx.x * kRedCols + 4 * ci;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < d) {
    for (int g = gi; g < parts; g += UN * kRedRows) {
      float4 v[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u)   // a part past the last reads the last one and is left out
        v[u] = *reinterpret_cast<const float4*>(part + (size_t)min(g + u * kRedRows, parts - 1) * d + c);
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        if (g + u * kRedRows >= parts) continue;
        s.x += v[u].x; s.y += v[u].y; s.z += v[u].z; s.w += v[u].w;
      }
    }
  }
  acc[gi][ci] = s;
  __syncthreads();
#pragma unroll
  for (int o = kRedRows / 2; o > 0; o >>= 1) {
    if (gi < o) {
      const float4 v = acc[gi + o][ci];
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
      acc[gi][ci] = s;
    }
    __syncthreads();
  }
  if (gi == 0 && c < d) {
    Elem<T>::store(dw, c, s.x);
    Elem<T>::store(dw, c + 1, s.y);
    Elem<T>::store(dw, c + 2, s.z);
    Elem<T>::store(dw, c + 3, s.w);
  }
}

// Workgroups of the backward kernel, and parts of dw: rows dealt evenly over
// the workgroups that are resident at once (8 waves a CU in bf16, 12 in
// binary32; 1024 at most). 16384 x 2048 bf16: 512 workgroups 48.4 us, 1024 50.7.
template <typename T> int norm_bwd_grid(int T_, int waves) {
  const int wg_waves = waves == 1 ? 4 : waves, rows = waves == 1 ? 4 : 1;
  const long resident = min(256 * ((sizeof(T) == 2 ? 8 : 12) / wg_waves), 1024) * rows;
  const long per = (T_ + resident - 1) / resident * rows;
  return static_cast<int>((T_ + per - 1) / per);
}

template <typename T, bool MX> int launch_norm(const NormArgs& a, hipStream_t s) {
  const bool stream = (long)a.T * a.d * sizeof(T) * (a.res ? 4 : 2) >= kStreamBytes;
  bool ok = true;
  norm_shape<T>(a.d, [&](auto w, auto u) {
    constexpr int W = w(), U = u();
    const int grid = W == 1 ? static_cast<int>((a.T + 3L) / 4) : a.T;
    if (!(ok = launchable(grid, kNormThreads<W>))) return;
    if (stream) add_rmsnorm_kernel<T, W, U, MX, true><<<grid, kNormThreads<W>, 0, s>>>(a);
    else add_rmsnorm_kernel<T, W, U, MX, false><<<grid, kNormThreads<W>, 0, s>>>(a);
  });
  MOE_CHECK_SUPPORTED(ok);
  return launch_status();
}

template <typename T> int launch_norm_bwd(const NormBwdArgs& a, void* dw, hipStream_t s) {
  const bool stream = (long)a.T * a.d * sizeof(T) * (a.dh ? 4 : 3) >= kStreamBytes;
  int grid = 0;
  norm_shape<T>(a.d, [&](auto w, auto u) {
    constexpr int W = w(), U = u();
    grid = norm_bwd_grid<T>(a.T, W);
    if (stream) rmsnorm_bwd_kernel<T, W, U, true><<<grid, kNormThreads<W>, 0, s>>>(a);
    else rmsnorm_bwd_kernel<T, W, U, false><<<grid, kNormThreads<W>, 0, s>>>(a);
  });
  if (int st = launch_status()) return st;
  if (!dw) return MOE_OK;
  norm_dw_kernel<T><<<(a.d + kRedCols - 1) / kRedCols, 1024, 0, s>>>(a.part, grid, a.d, static_cast<T*>(dw));
  return launch_status();
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_add_rmsnorm(int dtype, const void* x, const void* res, const void* w, int T, int d, float eps,
                               void* h, void* y, void* q, void* s, float* rstd, hipStream_t stream) {
  MOE_CHECK_ARG(valid_dtype(dtype) && T >= 0 && d > 0 && d % 8 == 0);
  MOE_CHECK_ARG(eps > 0.0f && eps < INFINITY);
  MOE_CHECK_SUPPORTED(d <= MOE_MAX_NORM_D);
  if (T == 0) return MOE_OK;   // tensors of no row may have no address
  MOE_CHECK_ARG((q == nullptr) == (s == nullptr) && (res == nullptr) == (h == nullptr));
  MOE_CHECK_ARG(q == nullptr || (dtype == MOE_BF16 && d % 128 == 0));
  MOE_CHECK_ARG(y != nullptr || q != nullptr);
  MOE_CHECK_ARG(x && w && aligned16(x) && aligned16(res) && aligned16(w) && aligned16(h) && aligned16(y));
  MOE_CHECK_ARG(aligned16(q) && aligned4(s) && aligned4(rstd));
  const NormArgs a{x, res, w, h, y, static_cast<uint8_t*>(q), static_cast<uint8_t*>(s), rstd, T, d, eps};
  if (dtype == MOE_F32) return launch_norm<float, false>(a, stream);
  return q ? launch_norm<uint16_t, true>(a, stream) : launch_norm<uint16_t, false>(a, stream);
}

extern "C" size_t moe_add_rmsnorm_bwd_workspace_bytes(int T, int d) {
  if (T < 1 || d < 1) return 0;
  // one row of parts per workgroup, whatever the type: at most 1024, or T
  return sizeof(float) * (size_t)min(T, 1024) * d;
}

extern "C" int moe_add_rmsnorm_bwd(int dtype, const void* dy, const void* h, const void* w, const float* rstd,
                                   const void* dh, int T, int d, void* dx, void* dw, void* ws, size_t ws_bytes,
                                   hipStream_t stream) {
  MOE_CHECK_ARG(valid_dtype(dtype) && T >= 0 && d > 0 && d % 8 == 0);
  MOE_CHECK_SUPPORTED(d <= MOE_MAX_NORM_D);
  MOE_CHECK_ARG(aligned16(dw));
  const bool rows = T > 0;
  MOE_CHECK_ARG(!rows || (dy && h && w && rstd && dx && aligned16(dy) && aligned16(h) && aligned16(w) &&
                          aligned4(rstd) && aligned16(dh) && aligned16(dx)));
  if (rows && dw != nullptr && (ws == nullptr || ws_bytes < moe_add_rmsnorm_bwd_workspace_bytes(T, d) || !aligned16(ws)))
    return MOE_ERR_WORKSPACE;
  if (!rows) {   // no row: dw is the empty sum
    if (dw == nullptr) return MOE_OK;
    const int grid = (d + kRedCols - 1) / kRedCols;
    if (dtype == MOE_F32) norm_dw_kernel<float><<<grid, 1024, 0, stream>>>(nullptr, 0, d, static_cast<float*>(dw));
    else norm_dw_kernel<uint16_t><<<grid, 1024, 0, stream>>>(nullptr, 0, d, static_cast<uint16_t*>(dw));
    return launch_status();
  }
  const NormBwdArgs a{dy, h, w, rstd, dh, dx, dw ? static_cast<float*>(ws) : nullptr, T, d};
  return dtype == MOE_F32 ? launch_norm_bwd<float>(a, dw, stream) : launch_norm_bwd<uint16_t>(a, dw, stream);
}
