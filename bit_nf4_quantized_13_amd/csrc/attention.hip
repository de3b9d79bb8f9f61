// Causal attention over packed sequences, forward and backward, on bf16 matrix
// instructions.  q [T x H x D], k, v [T x Hk x D]; head h reads the key-value
// head h / (H / Hk); row i attends to the rows j <= i of its own sequence:
//   s_ij = scale q_i k_j     lse_i = log sum_j e^s_ij     p_ij = e^(s_ij - lse_i)
//   o_i = sum_j p_ij v_j
//   dp_ij = do_i v_j         delta_i = sum_j p_ij dp_ij = do_i o_i
//   ds_ij = p_ij (dp_ij - delta_i) scale
//   dq_i = sum_j ds_ij k_j   dk_j = sum_i ds_ij q_i       dv_j = sum_i p_ij do_i
// (dk, dv over all heads of the group).  Rows of no sequence have o = 0,
// lse = -inf and no gradient.
//
// Bound: the matrix cores from a few hundred rows on (4 D operations a pair and
// head forward, 14 D backward: s and dp are formed twice so that every sum has
// one owner and a fixed order, no atomics), HBM below.
//
// All products are 32 x 32 x 16 with the score tile transposed so that its
// result layout is the next product's operand: the lane that receives score
// column n holds 16 of a 32-row tile's rows, 4 consecutive at a time, and the
// contraction over those rows may run in any order as long as both operands
// agree.  P goes from the accumulators to the operand in registers; the other
// operand, a tile stored by rows and needed by columns, is read from LDS with
// the transposing load.
//   forward  S' = K Q', O' += V' P'        (a lane owns one query: its softmax
//                                           maximum and sum are in the lane pair l, l ^ 32)
//   dq       S' = K Q', dP' = V dO', dQ' += K' dS'
//   dk, dv   S = Q K',  dP = dO V',  dV' += dO' P, dK' += Q' dS
// Scores, statistics, sums and gradients are fp32; P and dS are rounded to bf16
// for their product, which the matrix cores take no wider (relative 2^-9, as
// every stored input).  delta's o is taken with its rounding residual where the
// forward saved it, so that the bf16 of o does not enter dS.
//
// A workgroup is 4 waves with 32 rows each; the 64-row tiles of the other side
// are brought to LDS by direct transfers, one tile ahead.  Tile rows are 16-byte
// chunks in an order that depends on the row, so that both the row reads (one
// chunk of 16 rows) and the transposing reads (4 chunks of 4 rows) fall on all
// banks.  Head dimensions are padded to 64 or 128 with zeros in LDS.
//
// Workgroups find their tile without a list: sequence s owns the slots from
// start_s / 128 + s on, which is enough for its tiles whatever its start (128
// rows a tile); a workgroup looks its slot up among the starts, 64 at a time.
#include "launch.hpp"

namespace qnf4 {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kOwn = 32 * kWaves;  // rows a workgroup owns
constexpr int kStream = 64;        // rows of a tile that passes through LDS
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;

__device__ __forceinline__ uint32_t lds_addr(const void *p) { return (uint32_t)reinterpret_cast<uintptr_t>(p); }

__device__ __forceinline__ bf16x8 lds_frag(uint32_t addr) {
    __builtin_assume((addr & 15) == 0);
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const lds_u32x4 *>(addr));
}
// Lane i of 16 names row i / 4, columns 4 (i % 4) ..; it receives column i of the 4 rows.
__device__ __forceinline__ s16x4 lds_transposed(uint32_t addr) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4 *>(addr));
}
__device__ __forceinline__ bf16x8 join(s16x4 a, s16x4 b) {
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    const s16x8 v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, v);
}
__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
// Rows 8 s .. 8 s + 7 of an accumulator tile as bf16.
__device__ __forceinline__ bf16x8 operand_of(const f32x16 &t, int s) {
    uint4 w;
    w.x = pack_bf16x2(t[8 * s + 0], t[8 * s + 1]);
    w.y = pack_bf16x2(t[8 * s + 2], t[8 * s + 3]);
    w.z = pack_bf16x2(t[8 * s + 4], t[8 * s + 5]);
    w.w = pack_bf16x2(t[8 * s + 6], t[8 * s + 7]);
    return __builtin_bit_cast(bf16x8, w);
}
// The row of an accumulator tile that register i holds in half h of the wave.
__device__ __forceinline__ int tile_row(int i, int h) { return (i & 3) + 8 * (i >> 2) + 4 * h; }

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ float pair_max(float v) {
    const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
}
__device__ __forceinline__ float pair_sum(float v) {
    const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r.x) + __uint_as_float(r.y);
}

// The sequence rows [begin, end) and the first row of a workgroup's tile;
// outside: the rows belong to no sequence.  Segments: the rows before the
// first sequence, the sequences, the rows after the last.
struct Place {
    int begin, end, first;
    bool outside;
};
__device__ __forceinline__ int bound_at(const int32_t *cu, int S, int T, int i) {
    if (i <= 0) return 0;
    if (i >= S + 2) return T;
    const int c = cu[i - 1];
    return c < 0 ? 0 : c > T ? T : c;
}
__device__ __forceinline__ Place place_of(const int32_t *cu, int S, int T, int slot) {
    const int lane = threadIdx.x & 63;
    int lo = 0, len = S + 2;
    while (len > 1) {
        const int step = (len + 63) / 64, i = lo + lane * step;
        const bool before = lane * step < len && bound_at(cu, S, T, i) / kOwn + i <= slot;
        int n = __popcll(__ballot(before));
        n = n < 1 ? 1 : n;
        const int left = len - (n - 1) * step;
        lo += (n - 1) * step;
        len = step < left ? step : left;
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    Place p;
    p.begin = __builtin_amdgcn_readfirstlane(bound_at(cu, S, T, lo));
    p.end = __builtin_amdgcn_readfirstlane(bound_at(cu, S, T, lo + 1));
    p.first = p.begin + (slot - (p.begin / kOwn + lo)) * kOwn;
    p.outside = lo == 0 || lo == S + 1;
    return p;
}

// Tile layout in LDS: rows of DP bf16, chunk c of row r at chunk c ^ swizzle(r).
template <int DP>
__device__ __forceinline__ int swizzle(int r) {
    return DP == 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
}

// 16 bytes a lane from global memory to LDS: lane l writes dst + 16 l.
__device__ __forceinline__ void transfer16(__amdgpu_buffer_rsrc_t r, const void *dst, uint32_t voff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r, reinterpret_cast<__attribute__((address_space(3))) void *>(reinterpret_cast<uintptr_t>(dst)), 16, voff, 0, 0,
        0);
}

// The transfers of a wave: its quarter of a 64-row tile.
template <int DP>
struct Mover {
    static constexpr int kChunks = DP / 8, kRows = 64 / kChunks, kOps = kStream / kWaves / kRows;
    uint32_t voff[kOps];
    __device__ __forceinline__ void init(int64_t ld, int D) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
        for (int i = 0; i < kOps; ++i) {
            const int row = wave * (kStream / kWaves) + i * kRows + lane / kChunks;
            const int c = (lane % kChunks) ^ swizzle<DP>(row);
            // columns past D lie past every range: zeros
            voff[i] = c * 8 < D ? (uint32_t)(row * ld * 2 + c * 16) : 0x80000000u;
        }
    }
    // Rows [row0, row0 + 64) of x (pitch ld) to dst; zeros from row `end` on.
    __device__ __forceinline__ void load(const uint16_t *x, int64_t ld, int row0, int end, uint16_t *dst) const {
        int rows = end - row0;
        rows = rows < 0 ? 0 : rows > kStream ? kStream : rows;
        const __amdgpu_buffer_rsrc_t r = out_rsrc(x + (int64_t)row0 * ld, (int64_t)rows * ld * 2);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
        for (int i = 0; i < kOps; ++i) {
            const uint16_t *at = dst + (wave * (kStream / kWaves) + i * kRows) * DP;
            transfer16(r, at, voff[i]);
        }
    }
};

// Addresses inside a tile of what a lane reads: row fragments (32 rows, 16
// columns: row l % 32, columns 16 ks + 8 (l / 32) ..) and transposed fragments
// (32 columns from 32 dt, rows 16 s + 4 (l / 32) .. and 8 further).
template <int DP>
struct Reader {
    static constexpr int kSteps = DP / 16, kTiles = DP / 32;
    uint32_t row[kSteps], col[kTiles][2];
    __device__ __forceinline__ void init() {
        const int l = threadIdx.x & 63, h = l >> 5, r = l & 31, i = l & 15, g = (l >> 4) & 1;
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) row[ks] = r * DP * 2 + (((2 * ks + h) ^ swizzle<DP>(r)) * 16);
#pragma unroll
        for (int dt = 0; dt < kTiles; ++dt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int rr = 8 * u + 4 * h + i / 4, c = dt * 4 + g * 2 + (i & 3) / 2;
                col[dt][u] = rr * DP * 2 + ((c ^ swizzle<DP>(rr)) * 16) + (i & 1) * 8;
            }
    }
    // Rows 32 kt .. 32 kt + 31, column step ks.
    __device__ __forceinline__ bf16x8 rows(uint32_t tile, int kt, int ks) const {
        return lds_frag(tile + row[ks] + kt * 32 * DP * 2);
    }
    // Columns 32 dt .., row step s (rows 16 s .. 16 s + 15, in the accumulators' order).
    __device__ __forceinline__ bf16x8 cols(uint32_t tile, int dt, int s) const {
        return join(lds_transposed(tile + col[dt][0] + s * 16 * DP * 2),
                    lds_transposed(tile + col[dt][1] + s * 16 * DP * 2));
    }
};

// A wave's 32 rows as fragments in registers: row l % 32, zeros past `end` and D.
template <int DP>
__device__ __forceinline__ void load_rows(const uint16_t *x, int64_t ld, int row0, int end, int D, bf16x8 *f) {
    const int l = threadIdx.x & 63, row = row0 + (l & 31);
#pragma unroll
    for (int ks = 0; ks < DP / 16; ++ks) {
        const int c = 16 * ks + 8 * (l >> 5);
        uint4 w = make_uint4(0, 0, 0, 0);
        if (row < end && c < D) w = *reinterpret_cast<const uint4 *>(x + (int64_t)row * ld + c);
        f[ks] = __builtin_bit_cast(bf16x8, w);
    }
}

// Stores a transposed result (columns 32 dt + tile_row, row l % 32) times f as bf16 rows; res: the residuals.
template <int DP>
__device__ __forceinline__ void store_rows(uint16_t *y, uint16_t *res, int64_t ld, int row0, int end, int D,
                                           const f32x16 *t, float f) {
    const int l = threadIdx.x & 63, h = l >> 5, row = row0 + (l & 31);
    if (row >= end) return;
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const int c = 32 * dt + tile_row(i, h);
            if (c >= D) continue;
            const float a = t[dt][i] * f, b = t[dt][i + 1] * f, d = t[dt][i + 2] * f, e = t[dt][i + 3] * f;
            const uint2 w = make_uint2(pack_bf16x2(a, b), pack_bf16x2(d, e));
            *reinterpret_cast<uint2 *>(y + (int64_t)row * ld + c) = w;
            if (res) {
                const float ra = a - __uint_as_float(w.x << 16), rb = b - __uint_as_float(w.x & 0xFFFF0000u);
                const float rd = d - __uint_as_float(w.y << 16), re = e - __uint_as_float(w.y & 0xFFFF0000u);
                *reinterpret_cast<uint2 *>(res + (int64_t)row * ld + c) =
                    make_uint2(pack_bf16x2(ra, rb), pack_bf16x2(rd, re));
            }
        }
}

// Zeros in the rows [row0, end) of one head, by the whole workgroup.
__device__ __forceinline__ void zero_rows(uint16_t *y, int64_t ld, int row0, int end, int D) {
    const int chunks = D / 8;
    for (int i = threadIdx.x; i < kOwn * chunks; i += kThreads) {
        const int row = row0 + i / chunks;
        if (row < end) *reinterpret_cast<uint4 *>(y + (int64_t)row * ld + (i % chunks) * 8) = make_uint4(0, 0, 0, 0);
    }
}

// Workgroup -> head: neighbours in the grid (other XCDs) take other key-value
// heads, so that the heads of a group and the tiles of a head meet in one L2.
__device__ __forceinline__ int head_of(int p, int H, int Hk) { return (p % Hk) * (H / Hk) + p / Hk; }

template <int DP>
__global__ __launch_bounds__(kThreads) void attention_fwd_kernel(AttentionShape a, const uint16_t *__restrict__ q,
                                                                 const uint16_t *__restrict__ k,
                                                                 const uint16_t *__restrict__ v,
                                                                 const int32_t *__restrict__ cu,
                                                                 uint16_t *__restrict__ o, uint16_t *__restrict__ res,
                                                                 float *__restrict__ lse, int slots) {
    __shared__ __attribute__((aligned(16))) uint16_t ks_[2][kStream * DP], vs_[2][kStream * DP];
    const int head = head_of(blockIdx.x % a.H, a.H, a.Hk), kv = head / (a.H / a.Hk);
    // the long rows' tiles first
    const Place at = place_of(cu, a.S, a.T, slots - 1 - (int)(blockIdx.x / a.H));
    if (at.first >= at.end) return;
    const int64_t ldo = (int64_t)a.H * a.D;
    const int last = at.first + kOwn < at.end ? at.first + kOwn : at.end;
    if (at.outside) {
        zero_rows(o + head * a.D, ldo, at.first, last, a.D);
        if (res) zero_rows(res + head * a.D, ldo, at.first, last, a.D);
        for (int i = at.first + threadIdx.x; i < last; i += kThreads) lse[(int64_t)head * a.T + i] = -INFINITY;
        return;
    }
    const int l = threadIdx.x & 63, h = l >> 5, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row0 = at.first + 32 * wave, row = row0 + (l & 31);
    Mover<DP> mk, mv;
    mk.init(a.ldk, a.D);
    mv.init(a.ldv, a.D);
    Reader<DP> rd;
    rd.init();
    const uint16_t *kh = k + (int64_t)kv * a.D, *vh = v + (int64_t)kv * a.D;
    bf16x8 qf[DP / 16];
    load_rows<DP>(q + (int64_t)head * a.D, a.ldq, row0, at.end, a.D, qf);
    f32x16 acc[DP / 32];
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[dt][i] = 0.0f;
    float m = -INFINITY, sum = 0.0f;
    const float c = a.scale * kLog2e;
    const int tiles = (last - at.begin + kStream - 1) / kStream;
    mk.load(kh, a.ldk, at.begin, at.end, ks_[0]);
    mv.load(vh, a.ldv, at.begin, at.end, vs_[0]);
    for (int j = 0; j < tiles; ++j) {
        __syncthreads();  // tile j is in LDS, and nobody reads the other buffer
        const int key0 = at.begin + j * kStream;
        if (j + 1 < tiles) {
            mk.load(kh, a.ldk, key0 + kStream, at.end, ks_[(j + 1) & 1]);
            mv.load(vh, a.ldv, key0 + kStream, at.end, vs_[(j + 1) & 1]);
        }
        if (key0 > row0 + 31) continue;  // the wave's rows all come before this tile
        const uint32_t kt_ = lds_addr(ks_[j & 1]), vt_ = lds_addr(vs_[j & 1]);
        f32x16 s[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[t][i] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) s[t] = mfma(rd.rows(kt_, t, ks), qf[ks], s[t]);
        }
        if (key0 + kStream - 1 > row0) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (key0 + 32 * t + tile_row(i, h) > row) s[t][i] = -INFINITY;
        }
        float top = s[0][0];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
        top = pair_max(top);
        // the sums are moved to a new maximum only where one grew by more than 2^8: P
        // stays below 2^8, and no digits are lost in fp32 or bf16
        if (__ballot((top - m) * c > 8.0f)) {
            const float old = m;
            m = fmaxf(m, top);
            const float f = __builtin_amdgcn_exp2f((old - m) * c);
            sum *= f;
#pragma unroll
            for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[dt][i] *= f;
        }
        const float mc = m * c;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[t][i] = __builtin_amdgcn_exp2f(fmaf(s[t][i], c, -mc));
                sum += s[t][i];
            }
#pragma unroll
        for (int st = 0; st < 4; ++st) {
            const bf16x8 p = operand_of(s[st >> 1], st & 1);
#pragma unroll
            for (int dt = 0; dt < DP / 32; ++dt) acc[dt] = mfma(rd.cols(vt_, dt, st), p, acc[dt]);
        }
    }
    sum = pair_sum(sum);
    store_rows<DP>(o + head * a.D, res ? res + head * a.D : nullptr, ldo, row0, at.end, a.D, acc, 1.0f / sum);
    if (h == 0 && row < at.end) lse[(int64_t)head * a.T + row] = m * a.scale + logf(sum);
}

// dq, and delta for the dk, dv kernel.
template <int DP>
__global__ __launch_bounds__(kThreads) void attention_dq_kernel(
    AttentionShape a, const uint16_t *__restrict__ q, const uint16_t *__restrict__ k, const uint16_t *__restrict__ v,
    const uint16_t *__restrict__ o, const uint16_t *__restrict__ res, const float *__restrict__ lse,
    const uint16_t *__restrict__ dout, const int32_t *__restrict__ cu, uint16_t *__restrict__ dq, int64_t lddq,
    float *__restrict__ delta, int slots) {
    __shared__ __attribute__((aligned(16))) uint16_t ks_[2][kStream * DP], vs_[2][kStream * DP];
    const int head = head_of(blockIdx.x % a.H, a.H, a.Hk), kv = head / (a.H / a.Hk);
    const Place at = place_of(cu, a.S, a.T, slots - 1 - (int)(blockIdx.x / a.H));
    if (at.first >= at.end) return;
    const int64_t ldo = (int64_t)a.H * a.D;
    const int last = at.first + kOwn < at.end ? at.first + kOwn : at.end;
    if (at.outside) {
        zero_rows(dq + head * a.D, lddq, at.first, last, a.D);
        return;
    }
    const int l = threadIdx.x & 63, h = l >> 5, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row0 = at.first + 32 * wave, row = row0 + (l & 31);
    Mover<DP> mk, mv;
    mk.init(a.ldk, a.D);
    mv.init(a.ldv, a.D);
    Reader<DP> rd;
    rd.init();
    const uint16_t *kh = k + (int64_t)kv * a.D, *vh = v + (int64_t)kv * a.D;
    const int tiles = (last - at.begin + kStream - 1) / kStream;
    mk.load(kh, a.ldk, at.begin, at.end, ks_[0]);
    mv.load(vh, a.ldv, at.begin, at.end, vs_[0]);
    bf16x8 qf[DP / 16], df[DP / 16];
    load_rows<DP>(q + (int64_t)head * a.D, a.ldq, row0, at.end, a.D, qf);
    load_rows<DP>(dout + (int64_t)head * a.D, ldo, row0, at.end, a.D, df);
    float dl = 0.0f;
    {
        bf16x8 of[DP / 16];
        load_rows<DP>(o + (int64_t)head * a.D, ldo, row0, at.end, a.D, of);
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
            for (int e = 0; e < 8; ++e) dl += (float)df[ks][e] * (float)of[ks][e];
        if (res) {
            load_rows<DP>(res + (int64_t)head * a.D, ldo, row0, at.end, a.D, of);
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
                for (int e = 0; e < 8; ++e) dl += (float)df[ks][e] * (float)of[ks][e];
        }
    }
    dl = pair_sum(dl);
    const float ls = row < at.end ? lse[(int64_t)head * a.T + row] * kLog2e : INFINITY;
    if (h == 0 && row < at.end) delta[(int64_t)head * a.T + row] = dl;
    f32x16 acc[DP / 32];
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[dt][i] = 0.0f;
    const float c = a.scale * kLog2e;
    for (int j = 0; j < tiles; ++j) {
        __syncthreads();
        const int key0 = at.begin + j * kStream;
        if (j + 1 < tiles) {
            mk.load(kh, a.ldk, key0 + kStream, at.end, ks_[(j + 1) & 1]);
            mv.load(vh, a.ldv, key0 + kStream, at.end, vs_[(j + 1) & 1]);
        }
        const uint32_t kt_ = lds_addr(ks_[j & 1]), vt_ = lds_addr(vs_[j & 1]);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int k0 = key0 + 32 * t;
            if (k0 > row0 + 31) break;
            f32x16 s, dp;
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) {
                s = mfma(rd.rows(kt_, t, ks), qf[ks], s);
                dp = mfma(rd.rows(vt_, t, ks), df[ks], dp);
            }
            const bool edge = k0 + 31 > row0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float p = __builtin_amdgcn_exp2f(fmaf(s[i], c, -ls));
                if (edge && k0 + tile_row(i, h) > row) p = 0.0f;
                s[i] = p * (dp[i] - dl);
            }
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                const bf16x8 ds = operand_of(s, st);
#pragma unroll
                for (int dt = 0; dt < DP / 32; ++dt) acc[dt] = mfma(rd.cols(kt_, dt, 2 * t + st), ds, acc[dt]);
            }
        }
    }
    store_rows<DP>(dq + head * a.D, nullptr, lddq, row0, at.end, a.D, acc, a.scale);
}

// dk and dv of 128 keys of one key-value head: all rows after them, all heads of the group.
template <int DP>
__global__ __launch_bounds__(kThreads) void attention_dkv_kernel(
    AttentionShape a, const uint16_t *__restrict__ q, const uint16_t *__restrict__ k, const uint16_t *__restrict__ v,
    const float *__restrict__ lse, const float *__restrict__ delta, const uint16_t *__restrict__ dout,
    const int32_t *__restrict__ cu, uint16_t *__restrict__ dk, int64_t lddk, uint16_t *__restrict__ dv, int64_t lddv) {
    __shared__ __attribute__((aligned(16))) uint16_t qs_[2][kStream * DP], ds_[2][kStream * DP];
    __shared__ __attribute__((aligned(16))) float ls_[2][kStream], dl_[2][kStream];
    const int kv = blockIdx.x % a.Hk, group = a.H / a.Hk;
    const Place at = place_of(cu, a.S, a.T, (int)(blockIdx.x / a.Hk));  // the first keys have the most rows
    if (at.first >= at.end) return;
    const int64_t ldo = (int64_t)a.H * a.D;
    if (at.outside) {
        const int last = at.first + kOwn < at.end ? at.first + kOwn : at.end;
        zero_rows(dk + kv * a.D, lddk, at.first, last, a.D);
        zero_rows(dv + kv * a.D, lddv, at.first, last, a.D);
        return;
    }
    const int l = threadIdx.x & 63, h = l >> 5, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int key0 = at.first + 32 * wave, key = key0 + (l & 31);
    Mover<DP> mq, md;
    mq.init(a.ldq, a.D);
    md.init(ldo, a.D);
    Reader<DP> rd;
    rd.init();
    bf16x8 kf[DP / 16], vf[DP / 16];
    load_rows<DP>(k + (int64_t)kv * a.D, a.ldk, key0, at.end, a.D, kf);
    load_rows<DP>(v + (int64_t)kv * a.D, a.ldv, key0, at.end, a.D, vf);
    f32x16 ak[DP / 32], av[DP / 32];
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) ak[dt][i] = av[dt][i] = 0.0f;
    const float c = a.scale * kLog2e;
    const int per = (at.end - at.first + kStream - 1) / kStream, tiles = per * group;  // tiles of rows, head by head
    auto fetch = [&](int j) {
        const int hd = kv * group + j / per, r0 = at.first + (j % per) * kStream, b = j & 1;
        mq.load(q + (int64_t)hd * a.D, a.ldq, r0, at.end, qs_[b]);
        md.load(dout + (int64_t)hd * a.D, ldo, r0, at.end, ds_[b]);
        if (threadIdx.x < kStream) {  // a row past the end has lse = inf: p = 0
            const int r = r0 + threadIdx.x;
            const bool in = r < at.end;
            ls_[b][threadIdx.x] = in ? lse[(int64_t)hd * a.T + r] * kLog2e : INFINITY;
            dl_[b][threadIdx.x] = in ? delta[(int64_t)hd * a.T + r] : 0.0f;
        }
    };
    fetch(0);
    for (int j = 0; j < tiles; ++j) {
        __syncthreads();
        if (j + 1 < tiles) fetch(j + 1);
        const int r0 = at.first + (j % per) * kStream;
        const uint32_t qt_ = lds_addr(qs_[j & 1]), dt_ = lds_addr(ds_[j & 1]);
        const uint32_t lt_ = lds_addr(ls_[j & 1]) + 16 * h, et_ = lds_addr(dl_[j & 1]) + 16 * h;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int q0 = r0 + 32 * t;
            if (q0 + 31 < key0) continue;  // these rows all come before the wave's keys
            f32x16 s, dp;
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) {
                s = mfma(rd.rows(qt_, t, ks), kf[ks], s);
                dp = mfma(rd.rows(dt_, t, ks), vf[ks], dp);
            }
            const bool edge = q0 < key0 + 31;
            f32x16 p;
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const f32x4 ls = *reinterpret_cast<const lds_f32x4 *>(lt_ + (32 * t + 2 * i) * 4);
                const f32x4 dl = *reinterpret_cast<const lds_f32x4 *>(et_ + (32 * t + 2 * i) * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float pe = __builtin_amdgcn_exp2f(fmaf(s[i + e], c, -ls[e]));
                    if (edge && q0 + tile_row(i + e, h) < key) pe = 0.0f;
                    p[i + e] = pe;
                    s[i + e] = pe * (dp[i + e] - dl[e]);
                }
            }
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                const bf16x8 pb = operand_of(p, st), sb = operand_of(s, st);
#pragma unroll
                for (int dt = 0; dt < DP / 32; ++dt) {
                    av[dt] = mfma(rd.cols(dt_, dt, 2 * t + st), pb, av[dt]);
                    ak[dt] = mfma(rd.cols(qt_, dt, 2 * t + st), sb, ak[dt]);
                }
            }
        }
    }
    store_rows<DP>(dk + kv * a.D, nullptr, lddk, key0, at.end, a.D, ak, a.scale);
    store_rows<DP>(dv + kv * a.D, nullptr, lddv, key0, at.end, a.D, av, 1.0f);
}

int slots_of(const AttentionShape &a) { return a.T / kOwn + a.S + 2; }

}  // namespace

int64_t attention_groups(const AttentionShape &a) { return (int64_t)slots_of(a) * a.H; }

hipError_t launch_attention_fwd(const AttentionShape &a, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                                const int32_t *cu, uint16_t *o, uint16_t *res, float *lse, hipStream_t s) {
    const int slots = slots_of(a);
    const unsigned groups = (unsigned)slots * a.H;
    if (a.D <= 64)
        attention_fwd_kernel<64><<<groups, kThreads, 0, s>>>(a, q, k, v, cu, o, res, lse, slots);
    else
        attention_fwd_kernel<128><<<groups, kThreads, 0, s>>>(a, q, k, v, cu, o, res, lse, slots);
    return hipGetLastError();
}

hipError_t launch_attention_bwd(const AttentionShape &a, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                                const uint16_t *o, const uint16_t *res, const float *lse, const uint16_t *dout,
                                const int32_t *cu, uint16_t *dq, int64_t lddq, uint16_t *dk, int64_t lddk,
                                uint16_t *dv, int64_t lddv, float *delta, hipStream_t s) {
    const int slots = slots_of(a);
    const unsigned gq = (unsigned)slots * a.H, gk = (unsigned)slots * a.Hk;
    if (a.D <= 64)
        attention_dq_kernel<64><<<gq, kThreads, 0, s>>>(a, q, k, v, o, res, lse, dout, cu, dq, lddq, delta, slots);
    else
        attention_dq_kernel<128><<<gq, kThreads, 0, s>>>(a, q, k, v, o, res, lse, dout, cu, dq, lddq, delta, slots);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.D <= 64)
        attention_dkv_kernel<64><<<gk, kThreads, 0, s>>>(a, q, k, v, lse, delta, dout, cu, dk, lddk, dv, lddv);
    else
        attention_dkv_kernel<128><<<gk, kThreads, 0, s>>>(a, q, k, v, lse, delta, dout, cu, dk, lddk, dv, lddv);
    return hipGetLastError();
}

}  // namespace qnf4
