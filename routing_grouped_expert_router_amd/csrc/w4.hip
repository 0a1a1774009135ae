// The experts with 4-bit weights for single tokens and decode batches (gfx950):
//
//   H[s]  = silu(x[t] Wg[e]) * (x[t] Wu[e]),  s = (t, j) a slot, e its expert
//   y[t]  = y_add[t] + sum_j w[t,j] * (H[t,j] Wd[e])
//
// with every weight MXFP4 (OCP Microscaling v1.0: E2M1 elements, one E8M0 scale
// per 32 values along the contraction) laid out once by moe_w4_quantize in the
// order the matrix cores take it. Bound by the weights' bytes: a decode batch
// gives an expert a row or a few, so each weight is read once per launch and
// used for up to 64 rows. See include/moe.h for the contract.
//
// Layout. v_mfma_f32_16x16x32_bf16 takes, in lane l, eight K values of row
// l % 16 of its first operand. Which K values is free as long as both operands
// agree, so lane (n, g) holds the 32 consecutive values of scale block g of a
// 128-value step of column n: 16 bytes, one scale, four products. A wave reads
// 1 KB of consecutive bytes per 16 columns x 128 values, and a word per lane
// holds its scales for four such steps.
#include "mx_common.h"

namespace moe {

namespace {

typedef __attribute__((__vector_size__(8 * sizeof(__bf16)))) __bf16 w4bf16x8_t;
typedef __attribute__((__vector_size__(4 * sizeof(float)))) float w4f32x4_t;

constexpr int kTileN = 16;      // columns of a tile
constexpr int kStepK = 128;     // K values of a step
constexpr int kChunk = 4;       // steps that share a scale word
constexpr int kW4Threads = 256;

struct W4Mat {
  const uint8_t* q;
  const uint8_t* s;
};

// ------------------------------------------------------------------ quantise
// A workgroup stages 128 K values x 64 columns in LDS; thread (block g, column)
// turns 32 values into 16 code bytes and a scale byte.
constexpr int kQuantCols = 64, kQuantLdw = kQuantCols + 2;

__global__ void __launch_bounds__(kW4Threads) w4_quantize_kernel(const uint16_t* __restrict__ w, int K, int N,
                                                                 int tiles_c, uint8_t* __restrict__ q,
                                                                 uint8_t* __restrict__ s) {
  __shared__ uint16_t tile[kStepK * kQuantLdw];
  const int steps = K / kStepK, k5 = (steps + kChunk - 1) / kChunk;
  const int ct = blockIdx.x % tiles_c, kt = blockIdx.x / tiles_c % steps;
  const size_t m = blockIdx.x / tiles_c / steps;
  const int n0 = ct * kQuantCols, nv = min(kQuantCols, N - n0);
  const uint16_t* src = w + (m * K + (size_t)kt * kStepK) * N + n0;
  // N is a multiple of 16: pairs of columns never straddle its end
  for (int i = threadIdx.x; i < kStepK * kQuantCols / 2; i += kW4Threads) {
    const int r = i / (kQuantCols / 2), c = 2 * (i % (kQuantCols / 2));
    const uint32_t v = c < nv ? *reinterpret_cast<const uint32_t*>(src + (size_t)r * N + c) : 0u;
    *reinterpret_cast<uint32_t*>(tile + r * kQuantLdw + c) = v;
  }
  __syncthreads();
  const int c = threadIdx.x & 63, g = threadIdx.x >> 6;
  if (c >= nv) return;
  uint32_t v[16], mag = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint16_t* p = tile + (32 * g + 2 * i) * kQuantLdw + c;
    v[i] = p[0] | static_cast<uint32_t>(p[kQuantLdw]) << 16;
    mag = mag_max2(mag, v[i]);
  }
  // X = floor(log2 amax) - 2 (2 is the exponent of E2M1's largest value), -127 at least
  const int x = max(static_cast<int>(max_half(mag) >> 7) - 127 - 2, -127);
  const float scale = cvt_scale(x);
  V16 out;
#pragma unroll
  for (int i = 0; i < 4; ++i) {   // rounds to nearest even, saturates at 6
    uint32_t o = 0;
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, v[4 * i]), scale, 0);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, v[4 * i + 1]), scale, 1);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, v[4 * i + 2]), scale, 2);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, v[4 * i + 3]), scale, 3);
    out.w[i] = o;
  }
  const int n = n0 + c, lane = 16 * g + n % 16;
  const size_t t = m * (N / kTileN) + n / kTileN;
  *reinterpret_cast<V16*>(q + ((t * steps + kt) * 64 + lane) * 16) = out;
  uint8_t* sp = s + ((t * k5 + kt / kChunk) * 64 + lane) * 4;
  sp[kt % kChunk] = static_cast<uint8_t>(x + 127);
  if (kt == steps - 1)   // steps past K: zero
    for (int i = kt % kChunk + 1; i < kChunk; ++i) sp[i] = 0;
}

// ------------------------------------------------------------------ products
// The slots of the workgroup's expert, in slot order. Few slots (R <= E): unit
// u is a slot, and the first slot of each expert takes all of its expert's;
// else unit u is an expert. False: nothing to do. Every thread calls it.
struct Rows {
  int e, n;
};
MOE_DEV bool gather_rows(const int32_t* __restrict__ idx, int R, int E, int u, uint16_t* list, int* count, Rows& out) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int e = u;
  if (R <= E) {
    e = idx[u];
    if (e < 0 || e >= E) return false;
  }
  int n = 0, first = -1;
  for (int s0 = 0; s0 < R; s0 += kW4Threads) {
    const int s = s0 + tid;
    const bool hit = s < R && idx[s] == e;
    const uint64_t b = __ballot(hit);
    if (lane == 0) count[wave] = __popcll(b);
    __syncthreads();
    int at = n;
    for (int w = 0; w < kW4Threads / 64; ++w) {
      if (w < wave) at += count[w];
      n += count[w];
    }
    if (hit) list[at + __popcll(b & ((1ull << lane) - 1))] = static_cast<uint16_t>(s);
    __syncthreads();
  }
  if (n == 0) return false;
  first = list[0];
  if (R <= E && first != u) return false;
  out.e = e;
  out.n = n;
  return true;
}

// Eight bf16 values of one code word under scale byte `code`.
MOE_DEV w4bf16x8_t decode_w4(uint32_t w, float scale) {
  V16 v;
  v.w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
  v.w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
  v.w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
  v.w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  return __builtin_bit_cast(w4bf16x8_t, v);
}
MOE_DEV float w4_scale(uint32_t word, int step) {
  return __uint_as_float((word >> (8 * step) & 0xffu) << 23 | 0x400000u);
}

// Sums of NM matrices' 16-column tile over the wave's chunks of K, for RB
// blocks of 16 rows: acc[m][rb] holds, in lane (row r = lane % 16, g = lane / 16),
// columns 4g..4g+3 of row r. `row[rb]` is the lane's source row.
template <int NM, int RB>
MOE_DEV void w4_sums(const W4Mat (&mat)[NM], size_t tile, int K, int part, int parts, const uint16_t* const (&row)[RB],
                     w4f32x4_t (&acc)[NM][RB]) {
  const int lane = threadIdx.x & 63;
  const int steps = K / kStepK, chunks = (steps + kChunk - 1) / kChunk;
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int r = 0; r < RB; ++r) acc[m][r] = w4f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int c = part; c < chunks; c += parts) {
    uint32_t sw[NM];
    V16 qv[NM][kChunk];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      sw[m] = reinterpret_cast<const uint32_t*>(mat[m].s)[(tile * chunks + c) * 64 + lane];
#pragma unroll
      for (int i = 0; i < kChunk; ++i)   // a step past K reads the last one and is not used
        qv[m][i] = reinterpret_cast<const V16*>(mat[m].q)[(tile * steps + min(c * kChunk + i, steps - 1)) * 64 + lane];
    }
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      if (c * kChunk + i >= steps) break;   // wave-uniform
      V16 xv[RB][4];
#pragma unroll
      for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          xv[r][j] = reinterpret_cast<const V16*>(row[r])[(c * kChunk + i) * 16 + (lane >> 4) * 4 + j];
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const float scale = w4_scale(sw[m], i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const w4bf16x8_t a = decode_w4(qv[m][i].w[j], scale);
#pragma unroll
          for (int r = 0; r < RB; ++r)
            acc[m][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(w4bf16x8_t, xv[r][j]), acc[m][r], 0, 0, 0);
        }
      }
    }
  }
}

struct W4Args {
  const uint16_t* x;       // [T, d]
  const int32_t* idx;      // [R]
  const float* topk_w;     // [R]
  W4Mat wg, wu, wd;
  const uint16_t* y_add;   // [T, d] or null
  uint16_t* y;             // [T, d]
  uint16_t* h;             // [R, F] workspace
  float* part;             // [R, d] workspace: each slot's output row
  int T, d, E, k, F;
};

// WK waves share a tile's K, 4 / WK tiles per workgroup. Their sums meet in
// LDS and are added in the order of the parts.
template <bool GATE_UP, int WK, int RB>
MOE_DEV void w4_tile(const W4Args& a, const Rows& rows, int r0, int tile, bool valid, const uint16_t* list, float* red) {
  constexpr int NM = GATE_UP ? 2 : 1;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int part = wave % WK;
  const int K = GATE_UP ? a.d : a.F, N = GATE_UP ? a.F : a.d;
  const uint16_t* src[RB];
#pragma unroll
  for (int r = 0; r < RB; ++r) {   // a row past the last reads the last one; its sums are not stored
    const int s = list[min(r0 + 16 * r + (lane & 15), rows.n - 1)];
    src[r] = GATE_UP ? a.x + (size_t)(s / a.k) * K : a.h + (size_t)s * K;
  }
  w4f32x4_t acc[NM][RB];
  const size_t t = (size_t)rows.e * (N / kTileN) + tile;
  if (valid) {
    if constexpr (GATE_UP) {
      const W4Mat mat[2] = {a.wg, a.wu};
      w4_sums<2, RB>(mat, t, K, part, WK, src, acc);
    } else {
      const W4Mat mat[1] = {a.wd};
      w4_sums<1, RB>(mat, t, K, part, WK, src, acc);
    }
  }
  if constexpr (WK > 1) {
    // parts 1.. leave their sums, part 0 adds them
    __syncthreads();
    float4* slot = reinterpret_cast<float4*>(red) + (size_t)(wave - wave / WK - 1) * NM * RB * 64 + lane;
    if (valid && part > 0)
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int r = 0; r < RB; ++r) slot[(m * RB + r) * 64] = __builtin_bit_cast(float4, acc[m][r]);
    __syncthreads();
    if (!valid || part > 0) return;
    for (int p = 1; p < WK; ++p) {
      const float4* from = reinterpret_cast<const float4*>(red) + (size_t)(wave + p - wave / WK - 1) * NM * RB * 64 + lane;
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          const float4 v = from[(m * RB + r) * 64];
          acc[m][r] += w4f32x4_t{v.x, v.y, v.z, v.w};
        }
    }
  } else if (!valid) {
    return;
  }
  const int n = tile * kTileN + 4 * (lane >> 4);
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    const int at = r0 + 16 * r + (lane & 15);
    if (at >= rows.n) continue;
    const size_t o = (size_t)list[at] * N + n;
    if constexpr (GATE_UP) {
      float hv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) hv[i] = silu(acc[0][r][i]) * acc[1][r][i];
      // H is rounded once, to the type the next product's matrix cores take
      *reinterpret_cast<uint2*>(a.h + o) = make_uint2(pack_bf16x2(hv[0], hv[1]), pack_bf16x2(hv[2], hv[3]));
    } else {
      *reinterpret_cast<float4*>(a.part + o) = make_float4(acc[0][r][0], acc[0][r][1], acc[0][r][2], acc[0][r][3]);
    }
  }
}

// LDS: the slot list, then the parts' sums (up to 4 - 4 / WK waves of NM * RB
// tiles of 1 KB).
template <bool GATE_UP, int WK>
__global__ void __launch_bounds__(kW4Threads) w4_kernel(W4Args a) {
  constexpr int NM = GATE_UP ? 2 : 1, TN = 4 / WK, kManyRows = 4;
  __shared__ uint16_t list[MOE_W4_MAX_SLOTS];
  __shared__ int count[4];
  __shared__ __attribute__((aligned(16))) float red[WK > 1 ? (4 - TN) * NM * kManyRows * 256 : 4];
  const int R = a.T * a.k, N = GATE_UP ? a.F : a.d;
  const int tiles = N / kTileN, groups = (tiles + TN - 1) / TN;
  const int u = blockIdx.x / groups, tile = blockIdx.x % groups * TN + (threadIdx.x >> 6) / WK;
  Rows rows;
  if (!gather_rows(a.idx, R, a.E, u, list, count, rows)) return;
  const bool valid = tile < tiles;
  const int tc = valid ? tile : tiles - 1;
  if (rows.n <= 16) {
    w4_tile<GATE_UP, WK, 1>(a, rows, 0, tc, valid, list, red);
  } else {
    for (int r0 = 0; r0 < rows.n; r0 += 16 * kManyRows)
      w4_tile<GATE_UP, WK, kManyRows>(a, rows, r0, tc, valid, list, red);
  }
}

// y[t] = y_add[t] + sum_j w[t,j] part[t,j], slots without an expert left out.
__global__ void __launch_bounds__(256) w4_combine_kernel(W4Args a) {
  const int per = a.d / 4;
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long)a.T * per) return;
  const int t = static_cast<int>(i / per), c = static_cast<int>(i % per);
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (a.y_add) {
    const uint2 w = reinterpret_cast<const uint2*>(a.y_add + (size_t)t * a.d)[c];
    v[0] = __uint_as_float(w.x << 16);
    v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16);
    v[3] = __uint_as_float(w.y & 0xffff0000u);
  }
  for (int j = 0; j < a.k; ++j) {
    const size_t s = (size_t)t * a.k + j;
    const int e = a.idx[s];
    if (e < 0 || e >= a.E) continue;
    const float w = a.topk_w[s];
    const float4 p = reinterpret_cast<const float4*>(a.part + s * a.d)[c];
    v[0] = fmaf(w, p.x, v[0]);
    v[1] = fmaf(w, p.y, v[1]);
    v[2] = fmaf(w, p.z, v[2]);
    v[3] = fmaf(w, p.w, v[3]);
  }
  reinterpret_cast<uint2*>(a.y + (size_t)t * a.d)[c] = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

template <bool GATE_UP> int launch_w4(const W4Args& a, hipStream_t s) {
  const int K = GATE_UP ? a.d : a.F, N = GATE_UP ? a.F : a.d;
  const int chunks = (K / kStepK + kChunk - 1) / kChunk;
  const int wk = chunks >= 3 ? 4 : chunks;   // waves that share a tile's K: as many as it has chunks, up to 4
  const int tn = 4 / wk;
  const long units = min(a.T * a.k, a.E), grid = units * ((N / kTileN + tn - 1) / tn);
  MOE_CHECK_SUPPORTED(grid < (1L << 31));
  if (wk == 4) w4_kernel<GATE_UP, 4><<<(int)grid, kW4Threads, 0, s>>>(a);
  else if (wk == 2) w4_kernel<GATE_UP, 2><<<(int)grid, kW4Threads, 0, s>>>(a);
  else w4_kernel<GATE_UP, 1><<<(int)grid, kW4Threads, 0, s>>>(a);
  return launch_status();
}

// Workspace: H rows, then from a 16-byte boundary the slots' output rows.
size_t w4_part_offset(int T, int k, int F) { return ((size_t)T * k * F * 2 + 15) & ~static_cast<size_t>(15); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_w4_code_bytes(int K, int N) {
  return K > 0 && N > 0 ? (size_t)K * N / 2 : 0;
}

extern "C" size_t moe_w4_scale_bytes(int K, int N) {
  return K > 0 && N > 0 ? (size_t)((K + 511) / 512) * N * 16 : 0;
}

extern "C" int moe_w4_quantize(const void* w, int n_mat, int K, int N, void* q, void* s, hipStream_t stream) {
  MOE_CHECK_ARG(n_mat >= 0 && K > 0 && N > 0 && K % kStepK == 0 && N % kTileN == 0);
  if (n_mat == 0) return MOE_OK;
  MOE_CHECK_ARG(w && q && s && aligned16(w) && aligned16(q) && aligned4(s));
  const int tiles_c = (N + kQuantCols - 1) / kQuantCols;
  const long grid = (long)n_mat * tiles_c * (K / kStepK);
  MOE_CHECK_SUPPORTED(grid < (1L << 31));
  w4_quantize_kernel<<<(int)grid, kW4Threads, 0, stream>>>(static_cast<const uint16_t*>(w), K, N, tiles_c,
                                                          static_cast<uint8_t*>(q), static_cast<uint8_t*>(s));
  return launch_status();
}

extern "C" size_t moe_experts_w4_workspace_bytes(int T, int k, int d, int F) {
  if (T < 1 || k < 1 || d < 1 || F < 1) return 0;
  return w4_part_offset(T, k, F) + (size_t)T * k * d * sizeof(float);
}

extern "C" int moe_experts_w4(const moe_w4_desc* g, hipStream_t stream) {
  MOE_CHECK_ARG(g != nullptr);
  MOE_CHECK_ARG(g->T >= 0 && g->d > 0 && g->F > 0 && g->E >= 1 && g->k >= 1 && g->d % kStepK == 0 && g->F % kStepK == 0);
  MOE_CHECK_SUPPORTED(g->E <= MOE_MAX_EXPERTS && g->k <= MOE_MAX_TOPK && (long)g->T * g->k <= MOE_W4_MAX_SLOTS);
  if (g->T == 0) return MOE_OK;
  MOE_CHECK_ARG(g->x && g->topk_idx && g->topk_w && g->y && aligned16(g->x) && aligned16(g->y) && aligned16(g->y_add));
  MOE_CHECK_ARG(aligned4(g->topk_idx) && aligned4(g->topk_w));
  for (const moe_w4_tensor* w : {&g->w_gate, &g->w_up, &g->w_down})
    MOE_CHECK_ARG(w->q && w->s && aligned16(w->q) && aligned4(w->s));
  if (g->ws == nullptr || !aligned16(g->ws) || g->ws_bytes < moe_experts_w4_workspace_bytes(g->T, g->k, g->d, g->F))
    return MOE_ERR_WORKSPACE;
  auto mat = [](const moe_w4_tensor& t) { return W4Mat{static_cast<const uint8_t*>(t.q), static_cast<const uint8_t*>(t.s)}; };
  char* ws = static_cast<char*>(g->ws);
  const W4Args a{static_cast<const uint16_t*>(g->x), g->topk_idx, g->topk_w, mat(g->w_gate), mat(g->w_up), mat(g->w_down),
                 static_cast<const uint16_t*>(g->y_add), static_cast<uint16_t*>(g->y), reinterpret_cast<uint16_t*>(ws),
                 reinterpret_cast<float*>(ws + w4_part_offset(g->T, g->k, g->F)), g->T, g->d, g->E, g->k, g->F};
  if (int st = launch_w4<true>(a, stream)) return st;
  if (int st = launch_w4<false>(a, stream)) return st;
  w4_combine_kernel<<<(int)(((long)g->T * (g->d / 4) + 255) / 256), 256, 0, stream>>>(a);
  return launch_status();
}
