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

#include <type_traits>

namespace moe {

namespace {

typedef __attribute__((__vector_size__(8 * sizeof(__bf16)))) __bf16 w4bf16x8_t;
typedef __attribute__((__vector_size__(4 * sizeof(float)))) float w4f32x4_t;
typedef __attribute__((__vector_size__(4 * sizeof(uint32_t)))) uint32_t w4u32x4_t;

constexpr int kTileN = 16;      // columns of a tile
constexpr int kStepK = 128;     // K values of a step
constexpr int kChunk = 4;       // steps that share a scale word
constexpr int kW4Threads = 256;
// Slots an expert, on average, up to which a product goes 16 rows (8 of H's two
// terms) at a time: beyond, the kernel that shares decoded weights among more
// rows takes over, for gate/up later where its workgroups do not fill the chip.
// Measured (d 2048, F 1024, the call's time with few rows at a time against
// many): gate/up, 32 experts, 12 slots each, 38.0 us against 38.7, 16 slots 45
// against 41; 8 experts, 24 slots, 24.6 against 26.1, 32 slots 28.1 against
// 26.5. Down, 128 experts, 6 slots, 99 against 106, 8 slots 111 against 104; 32
// experts, 4 slots, 31.6 against 31.1, 6 slots 34.6 against 31.6; 8 experts, 8
// slots, 18.6 against 18.7, 12 slots 21.5 against 19.7.
constexpr int kFewRows = 12, kFewRowsSmall = 30, kFewRowsDown = 6;
// The down product and the weighted sum are one launch while few slots share
// an expert's weights, which that launch reads once a slot: up to half the
// experts, or up to two slots an expert where the caches keep the pool's down
// weights; 64 slots at most. Both products, one launch against two: 4 slots of
// 128 experts 9.7 us against 11.3, 16 slots 15.8 against 18.1, 64 slots 39.3
// against 42.1, 128 slots 65 against 58; 64 slots of 32 experts with 36 MB of
// down weights 28.2 against 28.4, with 143 MB 99 against 69; 8 experts, 32
// slots, 14.7 against 14.1.
inline bool sum_slots(int R, int E, long down_bytes) {
  return R <= 64 && (2 * R <= E || (R <= 2 * E && down_bytes <= (40L << 20)));
}
// Slots a workgroup, and parts of K (16 slots in all: 15.8 us with 4 a
// workgroup, 16.7 with 8).
constexpr int kW4SumSlots = 4, kW4SumParts = 4;

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

struct W4Args {
  const uint16_t* x;       // [T, d]
  const int32_t* idx;      // [R]
  const float* topk_w;     // [R]
  W4Mat wg, wu, wd;
  const uint16_t* y_add;   // [T, d] or null
  uint16_t* y;             // [T, d]
  uint16_t* h;             // [R, 2, F] workspace: each slot's hidden row in two terms
  float* part;             // [R, d] workspace: each slot's output row
  int T, d, E, k, F;
};

// Rows of the products' second operand: x as it is, H as two bf16 terms, the
// rounded value and what the rounding left (16 bits of H in all). One term
// alone, as the training layer's H is, would put its 2^-8 beside y's own (2.4e-3
// against 1.7e-3 relative). Up to eight rows the second term costs nothing: it
// takes the places of the sixteen that those rows leave.
template <bool GATE_UP> constexpr int kTerms = GATE_UP ? 1 : 2;
template <bool GATE_UP, typename V> MOE_DEV const V* w4_row(const W4Args& a, int s) {
  return reinterpret_cast<const V*>(GATE_UP ? a.x + (size_t)(s / a.k) * a.d : a.h + (size_t)s * 2 * a.F);
}

// A row's sums over H's two terms: lane i of sixteen has row i's first term,
// lane 8 + i its second.
MOE_DEV w4f32x4_t add_terms(w4f32x4_t v) {
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] += __shfl_xor(v[r], 8, 64);
  return v;
}

// Four columns of slot s, tile `tile`: H's two terms from the gate and up
// sums, or the slot's output.
template <bool GATE_UP, int NM>
MOE_DEV void w4_store(const W4Args& a, int s, int tile, const w4f32x4_t (&v)[NM]) {
  const int col = tile * kTileN + 4 * ((threadIdx.x & 63) >> 4);
  if constexpr (GATE_UP) {
    float hv[4], lo[4];
    uint32_t hi[2];
#pragma unroll
    for (int r = 0; r < 4; ++r) hv[r] = silu(v[0][r]) * v[1][r];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      hi[i] = pack_bf16x2(hv[2 * i], hv[2 * i + 1]);
      const float a0 = __uint_as_float(hi[i] << 16), a1 = __uint_as_float(hi[i] & 0xffff0000u);
      lo[2 * i] = __builtin_isfinite(a0) ? hv[2 * i] - a0 : 0.f;
      lo[2 * i + 1] = __builtin_isfinite(a1) ? hv[2 * i + 1] - a1 : 0.f;
    }
    uint16_t* row = a.h + (size_t)s * 2 * a.F + col;
    *reinterpret_cast<uint2*>(row) = make_uint2(hi[0], hi[1]);
    *reinterpret_cast<uint2*>(row + a.F) = make_uint2(pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]));
  } else {
    *reinterpret_cast<float4*>(a.part + (size_t)s * a.d + col) = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
  }
}

// Few rows an expert (a decode batch). 64 tokens, top-4 of 128 experts of
// 2048 x 1024: gate/up 44 us at 5.9 TB/s, down 26 us at 5.1, the weights' bytes
// and little else. One block of 16 rows at a time, whose chunk of x stays in
// registers while the wave runs down TPW column tiles, the next tile's codes
// in flight under the current one's products (that batch: 72 us with four
// tiles a wave, 89 with two, 107 with one). WK waves share K, so a workgroup
// covers 4 / WK groups of TPW tiles and its waves' sums meet in LDS once.
template <bool GATE_UP, int WK, int TPW, bool NT>
__global__ void __launch_bounds__(kW4Threads, 2) w4_few_kernel(W4Args a) {
  constexpr int NM = GATE_UP ? 2 : 1, TN = 4 / WK, NR = 16 / kTerms<GATE_UP>;   // rows at a time
  __shared__ uint16_t list[MOE_W4_MAX_SLOTS];
  __shared__ int count[4];
  __shared__ __attribute__((aligned(16))) float4 red[WK > 1 ? 4 * TPW * NM * 64 : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave % WK, grp = wave / WK;
  const int K = GATE_UP ? a.d : a.F, N = GATE_UP ? a.F : a.d;
  const int tiles = N / kTileN, groups = (tiles + TN * TPW - 1) / (TN * TPW);
  const int u = blockIdx.x / groups, tile0 = blockIdx.x % groups * TN * TPW + grp * TPW;
  Rows rows;
  if (!gather_rows(a.idx, a.T * a.k, a.E, u, list, count, rows)) return;
  const int steps = K / kStepK, chunks = (steps + kChunk - 1) / kChunk;
  const size_t t0 = (size_t)rows.e * tiles;
  const W4Mat mat[2] = {GATE_UP ? a.wg : a.wd, a.wu};
  for (int r0 = 0; r0 < rows.n; r0 += NR) {
    // a row past the last reads the last one; place NR + i of H's holds the second term of row i
    const int s = list[min(r0 + (lane & (NR - 1)), rows.n - 1)];
    const V16* src = w4_row<GATE_UP, V16>(a, s) + (lane >> 4) * 4 + (lane & 15) / NR * (K / 8);
    w4f32x4_t acc[TPW][NM];
#pragma unroll
    for (int i = 0; i < TPW; ++i)
#pragma unroll
      for (int m = 0; m < NM; ++m) acc[i][m] = w4f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int c = part; c < chunks; c += WK) {
      V16 qv[2][NM][kChunk];
      uint32_t sw[2][NM];
      auto fetch = [&](int i, V16 (&q)[NM][kChunk], uint32_t (&w)[NM]) {
        const size_t t = t0 + min(tile0 + i, tiles - 1);
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          w[m] = reinterpret_cast<const uint32_t*>(mat[m].s)[(t * chunks + c) * 64 + lane];
#pragma unroll
          for (int b = 0; b < kChunk; ++b)   // a step past K reads the last one and is not used
            q[m][b] = load16<NT>(mat[m].q + ((t * steps + min(c * kChunk + b, steps - 1)) * 64 + lane) * 16);
        }
      };
      fetch(0, qv[0], sw[0]);
      V16 xv[kChunk][4];
#pragma unroll
      for (int b = 0; b < kChunk; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) xv[b][j] = src[min(c * kChunk + b, steps - 1) * 16 + j];
      // every load of the first tile is issued before its first product
#pragma unroll
      for (int b = 0; b < kChunk; ++b) {
#pragma unroll
        for (int m = 0; m < NM; ++m) pin(qv[0][m][b]);
#pragma unroll
        for (int j = 0; j < 4; ++j) pin(xv[b][j]);
      }
#pragma unroll
      for (int i = 0; i < TPW; ++i) {
        if (i + 1 < TPW) fetch(i + 1, qv[(i + 1) & 1], sw[(i + 1) & 1]);
#pragma unroll
        for (int b = 0; b < kChunk; ++b) {
          if (c * kChunk + b >= steps) break;   // wave-uniform
#pragma unroll
          for (int m = 0; m < NM; ++m) {
            const float scale = w4_scale(sw[i & 1][m], b);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode_w4(qv[i & 1][m][b].w[j], scale),
                                                                  __builtin_bit_cast(w4bf16x8_t, xv[b][j]), acc[i][m], 0, 0, 0);
          }
        }
      }
    }
    const int at = r0 + (lane & 15);
    auto store = [&](int i, w4f32x4_t (&v)[NM]) {
      if constexpr (!GATE_UP) v[0] = add_terms(v[0]);
      if ((lane & 15) < NR && at < rows.n && tile0 + i < tiles) w4_store<GATE_UP>(a, list[at], tile0 + i, v);
    };
    if constexpr (WK == 1) {
#pragma unroll
      for (int i = 0; i < TPW; ++i) store(i, acc[i]);
    } else {
      if (r0 > 0) __syncthreads();   // the sums before are read
      float4* mine = red + (size_t)wave * TPW * NM * 64 + lane;
#pragma unroll
      for (int i = 0; i < TPW; ++i)
#pragma unroll
        for (int m = 0; m < NM; ++m) mine[(i * NM + m) * 64] = __builtin_bit_cast(float4, acc[i][m]);
      __syncthreads();
      for (int i = part; i < TPW; i += WK) {   // the group's waves share its tiles; parts are added in order
        w4f32x4_t v[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
          v[m] = w4f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int p = 0; p < WK; ++p)
            v[m] += __builtin_bit_cast(w4f32x4_t, red[((size_t)(grp * WK + p) * TPW * NM + i * NM + m) * 64 + lane]);
        }
        store(i, v);
      }
    }
  }
}

// Many rows an expert (short prompts, small pools). ROWS at a time, so that a
// decoded weight serves three or four products (48 rows of x, 32 of H in two
// terms; 64 of either are 3 to 30 % slower, fewer waves being at work). The rows'
// 128-value steps go through two LDS buffers that the four waves share, each
// wave runs down its own NT column tiles; rows of 256 bytes have their 16-byte
// chunks XOR-swizzled by the row, which spreads the 16 rows of a fragment over
// the banks. Row blocks are dealt to the workgroups of grid dimension y. 512
// tokens, top-4 of 8 experts of 2048 x 1024: 62 us for both products and the
// sum, 410 TFLOP/s (550 with H's second term counted), bound by the length of a
// step: with 64 rows and one term, 54 us, it took 46 without three quarters of
// the products, 47 without the loads, 54 without the decoding, and two steps a
// barrier, or loads two steps ahead, were slower (69, 56).
template <bool GATE_UP> constexpr int kManyRows = GATE_UP ? 48 : 32;
template <bool GATE_UP, int NT>
__global__ void __launch_bounds__(kW4Threads, 2) w4_many_kernel(W4Args a) {
  constexpr int NM = GATE_UP ? 2 : 1, ROWS = kManyRows<GATE_UP>, RB = ROWS / 16, NX = kTerms<GATE_UP>;
  __shared__ uint16_t list[MOE_W4_MAX_SLOTS];
  __shared__ int count[4];
  __shared__ w4u32x4_t xs[2][NX][ROWS * 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int K = GATE_UP ? a.d : a.F, N = GATE_UP ? a.F : a.d;
  const int tiles = N / kTileN, groups = (tiles + 4 * NT - 1) / (4 * NT);
  const int u = blockIdx.x / groups, tile0 = (blockIdx.x % groups * 4 + wave) * NT;
  Rows rows;
  if (!gather_rows(a.idx, a.T * a.k, a.E, u, list, count, rows)) return;
  const int steps = K / kStepK, chunks = (steps + kChunk - 1) / kChunk;
  const size_t t0 = (size_t)rows.e * tiles;
  const W4Mat mat[2] = {GATE_UP ? a.wg : a.wd, a.wu};
  const int sr = tid >> 4, sc = tid & 15;   // staging: rows sr + 16 i, chunk sc
  for (int r0 = blockIdx.y * ROWS; r0 < rows.n; r0 += gridDim.y * ROWS) {
    const w4u32x4_t* src[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {   // a row past the last reads the last one
      const int s = list[min(r0 + sr + 16 * i, rows.n - 1)];
      src[i] = w4_row<GATE_UP, w4u32x4_t>(a, s) + sc;
    }
    w4u32x4_t xv[NX][RB];
    V16 qv[NM][NT];
    uint32_t sv[NM][NT];
    auto fetch = [&](int st) {
#pragma unroll
      for (int x = 0; x < NX; ++x)
#pragma unroll
        for (int i = 0; i < RB; ++i) xv[x][i] = src[i][x * (K / 8) + st * 16];
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const size_t t = t0 + min(tile0 + i, tiles - 1);
          qv[m][i] = load16<false>(mat[m].q + ((t * steps + st) * 64 + lane) * 16);
          sv[m][i] = mat[m].s[((t * chunks + st / kChunk) * 64 + lane) * kChunk + st % kChunk];
        }
    };
    w4f32x4_t acc[NM][NT][RB];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r = 0; r < RB; ++r) acc[m][i][r] = w4f32x4_t{0.f, 0.f, 0.f, 0.f};
    __syncthreads();   // the block before is read
    fetch(0);
    for (int st = 0; st < steps; ++st) {
      w4u32x4_t(&buf)[NX][ROWS * 16] = xs[st & 1];
#pragma unroll
      for (int x = 0; x < NX; ++x)
#pragma unroll
        for (int i = 0; i < RB; ++i) buf[x][(sr + 16 * i) * 16 + (sc ^ sr)] = xv[x][i];
      V16 qc[NM][NT];
      float scale[NM][NT];
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          qc[m][i] = qv[m][i];
          scale[m][i] = w4_scale(sv[m][i], 0);
        }
      __syncthreads();   // one barrier a step: this buffer was last read two steps ago
      if (st + 1 < steps) fetch(st + 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w4bf16x8_t xf[NX][RB];
#pragma unroll
        for (int x = 0; x < NX; ++x)
#pragma unroll
          for (int r = 0; r < RB; ++r)
            xf[x][r] = __builtin_bit_cast(w4bf16x8_t, buf[x][(16 * r + (lane & 15)) * 16 + (((lane >> 4) * 4 + j) ^ (lane & 15))]);
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const w4bf16x8_t w = decode_w4(qc[m][i].w[j], scale[m][i]);
#pragma unroll
            for (int x = 0; x < NX; ++x)
#pragma unroll
              for (int r = 0; r < RB; ++r)
                acc[m][i][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, xf[x][r], acc[m][i][r], 0, 0, 0);
          }
      }
    }
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int at = r0 + 16 * r + (lane & 15);
      if (at >= rows.n) continue;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (tile0 + i >= tiles) continue;
        w4f32x4_t v[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) v[m] = acc[m][i][r];
        w4_store<GATE_UP>(a, list[at], tile0 + i, v);
      }
    }
  }
}

// The down product and the weighted sum at once, for a handful of slots. One
// token: 4.7 us, of which 2.7 are a launch's own and the weights' bytes 0.9. A
// workgroup takes 16 output columns, its waves the (slot, chunk of K) pairs in
// turn, the places of the product's rows all the same slot's H, first or second
// term. A slot's sums over K are added in order, then the token's slots.
constexpr int kOneWaves = 8;
__global__ void __launch_bounds__(64 * kOneWaves) w4_down_sum_kernel(W4Args a) {
  __shared__ float red[MOE_MAX_TOPK * kW4SumParts][kTileN];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int per = max(kW4SumSlots / a.k, 1), t0 = blockIdx.y * per, nt = min(per, a.T - t0);   // this workgroup's tokens
  const int R = nt * a.k, steps = a.F / kStepK, chunks = (steps + kChunk - 1) / kChunk, tiles = a.d / kTileN;
  const int parts = min(chunks, kW4SumParts);
  for (int it = wave; it < R * parts; it += kOneWaves) {
    const int s = t0 * a.k + it / parts, part = it % parts;
    const int e = a.idx[s];
    if (e < 0 || e >= a.E) continue;
    const size_t t = (size_t)e * tiles + blockIdx.x;
    const V16* src = w4_row<false, V16>(a, s) + (lane >> 4) * 4 + (lane & 15) / 8 * (a.F / 8);
    w4f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    for (int c = part; c < chunks; c += parts) {
      const uint32_t sw = reinterpret_cast<const uint32_t*>(a.wd.s)[(t * chunks + c) * 64 + lane];
      V16 qv[kChunk], xv[kChunk][4];
#pragma unroll
      for (int b = 0; b < kChunk; ++b) {
        const int st = min(c * kChunk + b, steps - 1);
        qv[b] = reinterpret_cast<const V16*>(a.wd.q)[(t * steps + st) * 64 + lane];
#pragma unroll
        for (int j = 0; j < 4; ++j) xv[b][j] = src[st * 16 + j];
      }
#pragma unroll
      for (int b = 0; b < kChunk; ++b) {
        if (c * kChunk + b >= steps) break;   // wave-uniform
        const float scale = w4_scale(sw, b);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode_w4(qv[b].w[j], scale), __builtin_bit_cast(w4bf16x8_t, xv[b][j]),
                                                        acc, 0, 0, 0);
      }
    }
    acc = add_terms(acc);
    if ((lane & 15) == 0)
#pragma unroll
      for (int r = 0; r < 4; ++r) red[it][4 * (lane >> 4) + r] = acc[r];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nt * kTileN; i += 64 * kOneWaves) {
    const int t = i / kTileN, c = i % kTileN;
    const size_t o = (size_t)(t0 + t) * a.d + blockIdx.x * kTileN + c;
    float v = a.y_add ? bf16_to_f32(a.y_add[o]) : 0.f;
    for (int j = 0; j < a.k; ++j) {
      const int s = (t0 + t) * a.k + j, e = a.idx[s];
      if (e < 0 || e >= a.E) continue;
      float p = 0.f;
      for (int q = 0; q < parts; ++q) p += red[(t * a.k + j) * parts + q][c];
      v = fmaf(a.topk_w[s], p, v);
    }
    a.y[o] = f32_to_bf16(v);
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
  constexpr int G = 4;   // slots whose loads are in flight together
  for (int j0 = 0; j0 < a.k; j0 += G) {
    int e[G];
    float w[G];
    float4 p[G];
#pragma unroll
    for (int j = 0; j < G; ++j) {   // a slot past k reads the last one and adds nothing
      const size_t s = (size_t)t * a.k + min(j0 + j, a.k - 1);
      e[j] = j0 + j < a.k ? a.idx[s] : -1;
      w[j] = a.topk_w[s];
      p[j] = reinterpret_cast<const float4*>(a.part + s * a.d)[c];
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
      if (e[j] < 0 || e[j] >= a.E) continue;
      v[0] = fmaf(w[j], p[j].x, v[0]);
      v[1] = fmaf(w[j], p[j].y, v[1]);
      v[2] = fmaf(w[j], p[j].z, v[2]);
      v[3] = fmaf(w[j], p[j].w, v[3]);
    }
  }
  reinterpret_cast<uint2*>(a.y + (size_t)t * a.d)[c] = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

template <bool GATE_UP, int WK, bool NT> void launch_few(const W4Args& a, long units, int tiles, hipStream_t s) {
  constexpr int TN = 4 / WK;
  // as many tiles a wave as leave four workgroups a CU
  auto grid = [&](int tpw) { return units * ((tiles + TN * tpw - 1) / (TN * tpw)); };
  if (grid(4) >= 1024) w4_few_kernel<GATE_UP, WK, 4, NT><<<(int)grid(4), kW4Threads, 0, s>>>(a);
  else if (grid(2) >= 1024) w4_few_kernel<GATE_UP, WK, 2, NT><<<(int)grid(2), kW4Threads, 0, s>>>(a);
  else w4_few_kernel<GATE_UP, WK, 1, NT><<<(int)grid(1), kW4Threads, 0, s>>>(a);
}
template <bool GATE_UP, bool NT> void launch_few(const W4Args& a, int wk, long units, int tiles, hipStream_t s) {
  if (wk == 4) launch_few<GATE_UP, 4, NT>(a, units, tiles, s);
  else if (wk == 2) launch_few<GATE_UP, 2, NT>(a, units, tiles, s);
  else launch_few<GATE_UP, 1, NT>(a, units, tiles, s);
}

template <bool GATE_UP> int launch_w4(const W4Args& a, hipStream_t s) {
  const int K = GATE_UP ? a.d : a.F, N = GATE_UP ? a.F : a.d, R = a.T * a.k, tiles = N / kTileN;
  const int chunks = (K / kStepK + kChunk - 1) / kChunk;
  const int wk = chunks >= 3 ? 4 : chunks;   // waves that share a tile's K: as many as it has chunks, up to 4
  const long units = min(R, a.E);
  auto groups_of = [&](int nt) { return (tiles + 4 * nt - 1) / (4 * nt); };
  const int few = !GATE_UP ? kFewRowsDown : units * groups_of(1) >= 512 ? kFewRows : kFewRowsSmall;
  if (R <= few * a.E) {
    const long bytes = units * 3 * a.d * (long)a.F * 17 / 32;
    // codes past the caches: 167 MB 47 us against 43, 372 MB 78 against 72, but
    // 53 MB, which three weight sets in turn leave in them, 19 against 21
    if (bytes >= kStreamBytes) launch_few<GATE_UP, true>(a, wk, units, tiles, s);
    else launch_few<GATE_UP, false>(a, wk, units, tiles, s);
  } else {
    auto many = [&](auto nt) {
      const long wg = units * groups_of(nt);
      const long blocks = (R + kManyRows<GATE_UP> - 1) / kManyRows<GATE_UP>, want = (1024 + wg - 1) / wg;   // four workgroups a CU
      w4_many_kernel<GATE_UP, nt><<<dim3((unsigned)wg, (unsigned)min(blocks, want)), kW4Threads, 0, s>>>(a);
    };
    using std::integral_constant;
    if constexpr (GATE_UP) {
      many(integral_constant<int, 1>());
    } else {
      // four tiles where their workgroups, over the rows there are, still cover
      // the CUs (512 tokens of 8 experts 61.6 us against 65.5 with two, 512 of
      // 32 74 against 80; 128 of 8 31.4 against 30.0, 128 of 32 40.0 against 38.9)
      if ((long)R * groups_of(4) >= 256L * kManyRows<GATE_UP>) many(integral_constant<int, 4>());
      else many(integral_constant<int, 2>());
    }
  }
  return launch_status();
}

// Workspace: H rows (two bf16 terms), then from a 16-byte boundary the slots' output rows.
size_t w4_part_offset(int T, int k, int F) { return ((size_t)T * k * F * 4 + 15) & ~static_cast<size_t>(15); }

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
  MOE_CHECK_SUPPORTED(launchable(grid, kW4Threads));
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
  // refused before anything is launched: no kernel takes more workgroups than
  // one for each 16 columns of each expert (or slot); the sum, a thread for four columns
  const long slots = (long)g->T * g->k, units = slots < g->E ? slots : g->E, cols = g->d > g->F ? g->d : g->F;
  MOE_CHECK_SUPPORTED(launchable(units * (cols / kTileN), 64 * kOneWaves));
  MOE_CHECK_SUPPORTED(launchable(((long)g->T * (g->d / 4) + 255) / 256, 256));
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
  if (sum_slots(g->T * g->k, g->E, (long)g->E * g->d * g->F * 17 / 32)) {
    const int per = g->k < kW4SumSlots ? kW4SumSlots / g->k : 1;
    w4_down_sum_kernel<<<dim3(g->d / kTileN, (g->T + per - 1) / per), 64 * kOneWaves, 0, stream>>>(a);
    return launch_status();
  }
  if (int st = launch_w4<false>(a, stream)) return st;
  w4_combine_kernel<<<(int)(((long)g->T * (g->d / 4) + 255) / 256), 256, 0, stream>>>(a);
  return launch_status();
}
