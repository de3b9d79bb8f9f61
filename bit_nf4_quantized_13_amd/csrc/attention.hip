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
// one owner and a fixed order, no atomics), HBM below.  Measured at D = 128: one
// sequence of 8192 rows, H / Hk = 32 / 8, forward 507 to 530 us a call (1.04 to 1.08 PFLOP/s),
// 537 to 591 in a trace of 20 (the matrix cores busy 54 % of the time, the exponentials and
// conversions between the products and the LDS reads beside them); 4 x 1024, 32 / 32, forward
// 59 to 68 us, dq 79 to 92, dk and dv 92 to 107 (0.5 to 0.7 PFLOP/s; least and median of 20).
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
// for their product, which the matrix cores take no wider (relative 2^-8, as
// every stored input).  Backward, the score products start from -lse / scale and
// the dp products from -delta, so that their results are the exponent and the
// second factor of ds at once.  delta's o is taken with its rounding residual where the
// forward saved it, so that the bf16 of o does not enter dS.
//
// A workgroup is 4 waves (or 8, in parts) with 32 rows each; the tiles of the other side
// are brought to LDS by direct transfers, one tile ahead.  Tile rows are 16-byte
// chunks in an order that depends on the row, so that both the row reads (one
// chunk of 16 rows) and the transposing reads (4 chunks of 4 rows) fall on all
// banks.  Head dimensions are padded to 64 or 128 with zeros in LDS.
//
// Workgroups find their tile without a list: sequence s owns the slots from
// start_s / OWN + s on, which is enough for its tiles whatever its start (OWN rows
// a tile); a workgroup looks its slot up among the starts, 64 at a time.
#include "launch.hpp"

namespace qnf4 {
namespace {

constexpr int kThreads = 256;      // of the kernel that adds partials
constexpr float kLog2e = 1.44269504088896340736f;

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
// The row of an accumulator tile that register i holds in the wave's lower half; the upper half's is 4 further.
__device__ __forceinline__ constexpr int tile_row(int i) { return (i & 3) + 8 * (i >> 2); }

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
template <int OWN>
__device__ __forceinline__ Place place_of(const int32_t *cu, int S, int T, int slot) {
    const int lane = threadIdx.x & 63;
    int lo = 0, len = S + 2, n, bound, step;
    do {
        step = (len + 63) / 64;
        const int i = lo + lane * step;
        bound = bound_at(cu, S, T, i);
        n = __popcll(__ballot(lane * step < len && bound / OWN + i <= slot));
        n = __builtin_amdgcn_readfirstlane(n < 1 ? 1 : n);
        const int left = len - (n - 1) * step;
        lo += (n - 1) * step;
        len = step < left ? step : left;
    } while (step > 1);
    Place p;  // the last step's lanes hold the segments' starts one by one
    p.begin = __builtin_amdgcn_readlane(bound, n - 1);
    p.end = n < 64 ? __builtin_amdgcn_readlane(bound, n) : __builtin_amdgcn_readfirstlane(bound_at(cu, S, T, lo + 1));
    p.first = p.begin + (slot - (p.begin / OWN + lo)) * OWN;
    p.outside = lo == 0 || lo == S + 1;
    return p;
}

// Tile layout in LDS: rows of DP bf16, chunk c of row r at chunk c ^ swizzle(r).
template <int DP>
__device__ __forceinline__ int swizzle(int r) {
    return DP == 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
}

// 16 (or 4) bytes a lane from global memory to LDS: lane l writes dst + 16 l (4 l).
__device__ __forceinline__ void transfer16(__amdgpu_buffer_rsrc_t r, uint32_t dst, uint32_t voff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r, reinterpret_cast<__attribute__((address_space(3))) void *>(dst), 16, voff, 0, 0, 0);
}
__device__ __forceinline__ void transfer4(__amdgpu_buffer_rsrc_t r, uint32_t dst, uint32_t voff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r, reinterpret_cast<__attribute__((address_space(3))) void *>(dst), 4, voff, 0, 0, 0);
}

// The barrier that hands a tile over: the wave's own transfers have arrived (a barrier
// orders LDS accesses, not transfers that are still on their way), then everybody's.
// Also where a wave has nothing to compute between its transfers and the barrier.
__device__ __forceinline__ void tile_barrier() {
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt 0
    __syncthreads();
}

// The transfers of a wave: its quarter of a tile of ROWS rows, kRows at a time.
// The chunk that a lane brings differs between its rows by an exclusive or with
// the row group's number.  KEEP: the offsets stay in registers over the kernel;
// otherwise two registers hold them and they are formed at every tile, for a
// kernel that has no registers left.
template <int DP, int ROWS, int WAVES, bool KEEP>
struct Mover {
    static constexpr int kChunks = DP / 8, kRows = 64 / kChunks, kOwnRows = ROWS / WAVES, kOps = kOwnRows / kRows;
    static constexpr uint32_t kNowhere = 0x80000000u;  // past every tile's range
    static_assert((int64_t)ROWS * kMaxPitch * 2 <= kNowhere, "a tile's rows, at the largest pitch");
    uint32_t base, chunk, off[KEEP ? kOps : 1];
    __device__ __forceinline__ uint32_t offset(uint32_t base, uint32_t chunk, int64_t ld, int D, int i) const {
        const uint32_t c = chunk ^ swizzle<DP>(i * kRows);
        return c * 8 < (uint32_t)D ? base + (uint32_t)(i * kRows * ld * 2) + c * 16 : kNowhere;
    }
    __device__ __forceinline__ void init(int64_t ld, int D) {
        const int lane = threadIdx.x & 63, row = (threadIdx.x >> 6) * kOwnRows + lane / kChunks;
        base = (uint32_t)(row * ld * 2);
        chunk = (lane % kChunks) ^ swizzle<DP>(row);
        if (KEEP) {
#pragma unroll
            for (int i = 0; i < kOps; ++i) off[i] = offset(base, chunk, ld, D, i);
        }
    }
    // Rows [row0, row0 + ROWS) of x (pitch ld) to dst; zeros from row `end` and column D on.
    __device__ __forceinline__ void load(const uint16_t *x, int64_t ld, int D, int row0, int end, uint32_t dst) const {
        int rows = end - row0;
        rows = rows < 0 ? 0 : rows > ROWS ? ROWS : rows;
        const __amdgpu_buffer_rsrc_t r = out_rsrc(x + (int64_t)row0 * ld, (int64_t)rows * ld * 2);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        uint32_t b = base, ch = chunk;
        if (!KEEP) asm volatile("" : "+v"(b), "+v"(ch));  // formed here, not kept over the kernel's loop
#pragma unroll
        for (int i = 0; i < kOps; ++i)
            transfer16(r, dst + (wave * kOwnRows + i * kRows) * DP * 2,
                       KEEP ? off[KEEP ? i : 0] : offset(b, ch, ld, D, i));
    }
};

// What a lane reads of a tile: row fragments (32 rows, 16 columns: row l % 32,
// columns 16 ks + 8 (l / 32) ..) and transposed fragments (32 columns from 32
// dt, rows 16 s + 4 (l / 32) .. and 8 further).  The chunk order is an exclusive
// or, so every step's address is the lane's first one with a constant xored in
// (tiles start at multiples of their row size).  KEEP: the steps' addresses stay
// in registers, with the tile and the rows as the instructions' offsets.
template <int DP, bool KEEP>
struct Reader {
    static constexpr int kSteps = DP / 16, kTiles = DP / 32, kRow = DP * 2;
    uint32_t row0, col0, row[KEEP ? kSteps : 1], col[KEEP ? kSteps : 1];
    // first: of the tile's rows, a multiple of 32
    __device__ __forceinline__ void init(int first) {
        const int l = threadIdx.x & 63, h = l >> 5, r = l & 31, i = l & 15, g = (l >> 4) & 1;
        row0 = (first + r) * kRow + (h ^ swizzle<DP>(r)) * 16;
        const int rr = 4 * h + i / 4;
        col0 = (first + rr) * kRow + ((g * 2 + (i & 3) / 2) ^ swizzle<DP>(rr)) * 16 + (i & 1) * 8;
        if (KEEP) {
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) {
                row[ks] = row0 ^ (ks * 32);
                col[ks] = col0 ^ (ks * 32);
            }
        }
    }
    // Rows 32 kt .. 32 kt + 31, column step ks.
    __device__ __forceinline__ bf16x8 rows(uint32_t tile, int kt, int ks) const {
        const uint32_t at = KEEP ? row[KEEP ? ks : 0] + tile : (tile + row0) ^ (ks * 32);
        return lds_frag(at + kt * 32 * kRow);
    }
    // Columns 32 dt .., row step s (rows 16 s .. 16 s + 15, in the accumulators' order).
    __device__ __forceinline__ bf16x8 cols(uint32_t tile, int dt, int s) const {
        const uint32_t a = KEEP ? col[KEEP ? 2 * dt : 0] + tile : (tile + col0) ^ (dt * 64);
        const uint32_t b = KEEP ? col[KEEP ? 2 * dt + 1 : 0] + tile : (tile + col0) ^ (dt * 64 + 32);
        return join(lds_transposed(a + s * 16 * kRow), lds_transposed(b + s * 16 * kRow + 8 * kRow));
    }
};

// NaN and infinity keep to the causal order.  A masked p or ds is 0, but its product still
// meets the other operand's row, and 0 times NaN is NaN.  So a workgroup whose results are
// not all finite forms them once more, in a loop of its own: tiles that have masked places
// enter those products with their finite values alone, and what the others give to the
// rows that take them is added to the stored results (a running sum: the order is
// causal).  Finite results have the same bits either way; where all are finite this
// costs the look at them (us, without / with: 8192 rows forward 507 / 512, 4 x 1024 forward
// and backward 228 / 232, (700, 3, 517, 1, 250, 1025) 12 / 4 D 64 62 / 64).  With one NaN in v
// 4 x 1024 takes 395, with NaN throughout 680.
template <int N>
__device__ __forceinline__ bool not_finite(const f32x16 *t) {
    float z[N] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int dt = 0; dt < N; ++dt) z[dt] = fmaf(t[dt][i], 0.0f, z[dt]);
#pragma unroll
    for (int dt = 1; dt < N; ++dt) z[0] += z[dt];
    return z[0] != z[0];
}
// A tile of COUNT elements to another place in LDS (or its own), by the whole workgroup;
// finite_only: zeros for the others.
template <int COUNT>
__device__ __forceinline__ void copy_tile(uint32_t to, uint32_t from, bool finite_only) {
#pragma unroll 1
    for (int i = threadIdx.x; i < COUNT / 8; i += blockDim.x) {
        u32x4 w = *reinterpret_cast<const lds_u32x4 *>(from + i * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (finite_only && (w[e] & 0x7F80u) == 0x7F80u) w[e] &= 0xFFFF0000u;
            if (finite_only && (w[e] & 0x7F800000u) == 0x7F800000u) w[e] &= 0xFFFFu;
        }
        *reinterpret_cast<lds_u32x4 *>(to + i * 16) = w;
    }
}
// One wave: adds to its stored rows [first, last) of y, two columns a lane, what is not
// finite in the rows of x that they take: those from `start` up to the row itself, or (DOWN)
// from the row itself up to `start`, which is left out; of `heads` matrices, D columns
// apart.  Weights are positive, so that an infinity keeps its sign; SIGNED: NaN instead.
template <bool DOWN, bool SIGNED, typename Y>
__device__ __forceinline__ void add_not_finite(Y *y, int64_t ldy, int first, int last, const uint16_t *x, int64_t ldx,
                                               int heads, int start, int D) {
    __builtin_amdgcn_s_waitcnt(0x0F70);  // the rows are stored
    __threadfence_block();
    const int c = 2 * (threadIdx.x & 63);
    if (c >= D) return;
    auto term = [](uint32_t bits) {
        return (bits & 0x7F800000u) != 0x7F800000u ? 0.0f : SIGNED ? NAN : __uint_as_float(bits);
    };
    float sum0 = 0.0f, sum1 = 0.0f;
    const int rows = DOWN ? start - first : last - start;
#pragma unroll 1
    for (int n = 0; n < rows; ++n) {
        const int i = DOWN ? start - 1 - n : start + n;
#pragma unroll 1
        for (int hd = 0; hd < heads; ++hd) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(x + (int64_t)i * ldx + hd * D + c);
            sum0 += term(w << 16);
            sum1 += term(w & 0xFFFF0000u);
        }
        if (i < first || i >= last || (sum0 == 0.0f && sum1 == 0.0f)) continue;
        Y *at = y + (int64_t)i * ldy + c;
        if constexpr (sizeof(Y) == 2) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(at);
            *reinterpret_cast<uint32_t *>(at) =
                pack_bf16x2(__uint_as_float(w << 16) + sum0, __uint_as_float(w & 0xFFFF0000u) + sum1);
        } else {
            at[0] += sum0;
            at[1] += sum1;
        }
    }
}

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

// A wave's transposed result (columns 32 dt + tile_row + 4 (l / 32), row l % 32) on its
// way to memory: a lane holds 4 values of a row here and there, so the tile goes
// through the wave's own LDS (32 rows of DP bf16, chunks of 16 bytes in an order that
// depends on the row) and leaves as whole rows (8-byte pieces from the registers cost the
// forward of 4 x 1024, 32 heads, 69 us against 63).
template <int DP>
struct RowWriter {
    static constexpr int kChunks = DP / 8, kRows = 64 / kChunks;
    typedef u32x2 pair __attribute__((may_alias));
    typedef u32x4 chunk __attribute__((may_alias));
    char *lds;
    static __device__ __forceinline__ int order(int r) { return DP == 128 ? r & 15 : (r >> 1) & 7; }
    __device__ __forceinline__ void put(int dt, int i, uint32_t w0, uint32_t w1) const {
        const int l = threadIdx.x & 63, r = l & 31;
        *reinterpret_cast<pair *>(lds + r * DP * 2 + (((4 * dt + i / 4) ^ order(r)) * 16) + (l >> 5) * 8) = u32x2{w0, w1};
    }
    __device__ __forceinline__ void out(uint16_t *y, int64_t ld, int row0, int end, int D) const {
        const int l = threadIdx.x & 63, c = l % kChunks;
        asm volatile("" ::: "memory");  // the wave's own writes come first: LDS keeps their order
#pragma unroll
        for (int j = 0; j < 32 / kRows; ++j) {
            const int r = j * kRows + l / kChunks;
            const u32x4 w = *reinterpret_cast<const chunk *>(lds + r * DP * 2 + ((c ^ order(r)) * 16));
            if (row0 + r < end && c * 8 < D) *reinterpret_cast<chunk *>(y + (int64_t)(row0 + r) * ld + c * 8) = w;
        }
        asm volatile("" ::: "memory");
    }
};

// The result times f as bf16 rows; res: what the rounding drops.  lds: the wave's 64 DP bytes.
template <int DP>
__device__ __forceinline__ void store_rows(void *lds, uint16_t *y, uint16_t *res, int64_t ld, int row0, int end, int D,
                                           const f32x16 *t, float f) {
    const RowWriter<DP> to{static_cast<char *>(lds)};
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            to.put(dt, i, pack_bf16x2(t[dt][i] * f, t[dt][i + 1] * f), pack_bf16x2(t[dt][i + 2] * f, t[dt][i + 3] * f));
    to.out(y, ld, row0, end, D);
    if (!res) return;
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float a = t[dt][i] * f, b = t[dt][i + 1] * f, c = t[dt][i + 2] * f, d = t[dt][i + 3] * f;
            const uint32_t w = pack_bf16x2(a, b), x = pack_bf16x2(c, d);
            to.put(dt, i, pack_bf16x2(a - __uint_as_float(w << 16), b - __uint_as_float(w & 0xFFFF0000u)),
                   pack_bf16x2(c - __uint_as_float(x << 16), d - __uint_as_float(x & 0xFFFF0000u)));
        }
    to.out(res, ld, row0, end, D);
}

// Zeros in the rows [row0, end) of one head, by the whole workgroup.
template <int OWN>
__device__ __forceinline__ void zero_rows(uint16_t *y, int64_t ld, int row0, int end, int D) {
    const int chunks = D / 8;
    for (int i = threadIdx.x; i < OWN * chunks; i += blockDim.x) {
        const int row = row0 + i / chunks;
        if (row < end) *reinterpret_cast<uint4 *>(y + (int64_t)row * ld + (i % chunks) * 8) = make_uint4(0, 0, 0, 0);
    }
}

// Workgroup -> head: neighbours in the grid (other XCDs) take other key-value
// heads, so that the heads of a group and the tiles of a head meet in one L2.
__device__ __forceinline__ int head_of(int p, int H, int Hk) { return (p % Hk) * (H / Hk) + p / Hk; }

// A workgroup's waves: GROUPS of 32 rows, each group in PARTS.  Where there are few
// workgroups, the parts share their group's rows, each with its own rows of every tile,
// and their results meet in LDS at the end: a lane's registers, 64 apart.
template <int DP, int PARTS, int GROUPS>
struct Team {
    static constexpr int kFloats = DP / 2 * 64;  // of a wave's accumulators
    int lane, wave, group, part;
    __device__ __forceinline__ Team() {
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        group = wave % GROUPS;
        part = wave / GROUPS;
    }
    // Where a part's results wait for the one that adds them: slot 0 .. PARTS - 2.
    __device__ __forceinline__ float *slot(void *lds, int i) const {
        return static_cast<float *>(lds) + (i * GROUPS + group) * kFloats;
    }
};
template <int N>
__device__ __forceinline__ void put_tiles(float *to, const f32x16 *t) {
#pragma unroll
    for (int dt = 0; dt < N; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) to[(dt * 16 + i) * 64] = t[dt][i];
}
template <int N>
__device__ __forceinline__ void add_tiles(f32x16 *t, float f, const float *from, float g) {
#pragma unroll
    for (int dt = 0; dt < N; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) t[dt][i] = t[dt][i] * f + from[(dt * 16 + i) * 64] * g;
}

template <int DP, int PARTS, int GROUPS>
__global__ __launch_bounds__(64 * PARTS * GROUPS, 2) void attention_fwd_kernel(AttentionShape a, const uint16_t *__restrict__ q,
                                                                 const uint16_t *__restrict__ k,
                                                                 const uint16_t *__restrict__ v,
                                                                 const int32_t *__restrict__ cu,
                                                                 uint16_t *__restrict__ o, uint16_t *__restrict__ res,
                                                                 float *__restrict__ lse, int slots) {
    constexpr int OWN = 32 * GROUPS, kShare = GROUPS == 4 ? 64 : 32, kStep = kShare * PARTS;  // rows of a tile: a part's, all
    __shared__ __attribute__((aligned(256))) uint16_t tiles_[4][kStep * DP];
    uint16_t(*ks_)[kStep * DP] = tiles_, (*vs_)[kStep * DP] = tiles_ + 2;
    __shared__ float meet[2][PARTS > 1 ? 64 * PARTS * GROUPS : 1];
    __shared__ int odd;  // a result is not finite
    const int head = head_of(blockIdx.x % a.H, a.H, a.Hk), kv = head / (a.H / a.Hk);
    // from the last rows back: of one sequence, those with the most keys first
    const Place at = place_of<OWN>(cu, a.S, a.T, slots - 1 - (int)(blockIdx.x / a.H));
    if (at.first >= at.end) return;
    const int64_t ldo = (int64_t)a.H * a.D;
    const int last = at.first + OWN < at.end ? at.first + OWN : at.end;
    if (at.outside) {
        zero_rows<OWN>(o + head * a.D, ldo, at.first, last, a.D);
        if (res) zero_rows<OWN>(res + head * a.D, ldo, at.first, last, a.D);
        for (int i = at.first + threadIdx.x; i < last; i += blockDim.x) lse[(int64_t)head * a.T + i] = -INFINITY;
        return;
    }
    const Team<DP, PARTS, GROUPS> team;
    const int l = team.lane, h = l >> 5, part = team.part, row0 = at.first + 32 * team.group, row = row0 + (l & 31);
    Mover<DP, kStep, PARTS * GROUPS, true> mk, mv;
    mk.init(a.ldk, a.D);
    mv.init(a.ldv, a.D);
    Reader<DP, true> rd;
    rd.init(kShare * part);
    const uint16_t *kh = k + (int64_t)kv * a.D, *vh = v + (int64_t)kv * a.D;
    bf16x8 qf[DP / 16];
    load_rows<DP>(q + (int64_t)head * a.D, a.ldq, row0, at.end, a.D, qf);
    f32x16 acc[DP / 32];
    float m, sum;
    const float c = a.scale * kLog2e;
    const int tiles = (last - at.begin + kStep - 1) / kStep;
    auto load = [&](int tile0, int b) {
        mk.load(kh, a.ldk, a.D, tile0, at.end, lds_addr(ks_[b]));
        mv.load(vh, a.ldv, a.D, tile0, at.end, lds_addr(vs_[b]));
    };
    auto start = [&] {
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[dt][i] = 0.0f;
        m = -INFINITY;
        sum = 0.0f;
    };
    auto products = [&](int tile0, const uint32_t kt_, const uint32_t vt_) __attribute__((always_inline)) {
        const int key0 = tile0 + kShare * part;
        if (key0 > row0 + 31) return;  // the wave's rows all come before this tile
        f32x16 s[kShare / 32];
#pragma unroll
        for (int t = 0; t < kShare / 32; ++t) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[t][i] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) s[t] = mfma(rd.rows(kt_, t, ks), qf[ks], s[t]);
        }
        if (key0 + kShare - 1 > row0) {
#pragma unroll
            for (int t = 0; t < kShare / 32; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (key0 + 32 * t + tile_row(i) > row - 4 * h) s[t][i] = -INFINITY;
        }
        float top = s[0][0];
#pragma unroll
        for (int t = 0; t < kShare / 32; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
        top = pair_max(top);
        // the sums are moved to a new maximum only where one grew by more than 2^8: P
        // stays below 2^8, and no digits are lost in fp32 or bf16
        if (__ballot((top - m) * c > 8.0f)) {
            const float old = m;
            m = fmaxf(m, top);
            // no score above -inf yet: no key that the row attends to met by this part, or scores of -inf
            const float f = m == old ? 1.0f : __builtin_amdgcn_exp2f((old - m) * c);
            sum *= f;
#pragma unroll
            for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[dt][i] *= f;
        }
        const float mc = fmaxf(m * c, -0x1.fffffep127f);  // finite: p is 0 under it
#pragma unroll
        for (int t = 0; t < kShare / 32; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[t][i] = __builtin_amdgcn_exp2f(fmaf(s[t][i], c, -mc));
                sum += s[t][i];
            }
#pragma unroll
        for (int st = 0; st < kShare / 16; ++st) {
            const bf16x8 p = operand_of(s[st >> 1], st & 1);
#pragma unroll
            for (int dt = 0; dt < DP / 32; ++dt) acc[dt] = mfma(rd.cols(vt_, dt, st), p, acc[dt]);
        }
    };
    // B: the buffer that tile j is in, a constant so that it is part of the instructions' offsets
    auto tile_step = [&](int j, auto buf) {
        constexpr int B = decltype(buf)::value;
        tile_barrier();  // tile j is in LDS, and nobody reads the other buffer
        const int tile0 = at.begin + j * kStep;
        if (j + 1 < tiles) load(tile0 + kStep, 1 - B);
        products(tile0, lds_addr(ks_[B]), lds_addr(vs_[B]));
    };
    if (threadIdx.x == 0) odd = 0;
    load(at.begin, 0);
    start();
    for (int j = 0; j < tiles; j += 2) {
        tile_step(j, std::integral_constant<int, 0>());
        if (j + 1 < tiles) tile_step(j + 1, std::integral_constant<int, 1>());
    }
    if (not_finite<DP / 32>(acc)) odd = 1;
    tile_barrier();  // the tiles are read
    const bool ordered = odd;
    if (ordered) {
        start();
#pragma unroll 1
        for (int j = 0; j < tiles; ++j) {
            const int tile0 = at.begin + j * kStep;
            load(tile0, 0);
            tile_barrier();
            if (tile0 + kStep > at.first) {
                copy_tile<kStep * DP>(lds_addr(vs_[0]), lds_addr(vs_[0]), true);
                __syncthreads();
            }
            products(tile0, lds_addr(ks_[0]), lds_addr(vs_[0]));
            __syncthreads();
        }
    }
    sum = pair_sum(sum);
    float *mine = team.slot(tiles_, 0);
    if (PARTS > 1) {
        if (part > 0) put_tiles<DP / 32>(team.slot(tiles_, part - 1) + l, acc);
        meet[0][threadIdx.x] = m;
        meet[1][threadIdx.x] = sum;
        __syncthreads();
        if (part > 0) return;
#pragma unroll
        for (int p = 1; p < PARTS; ++p) {
            const int other = threadIdx.x + 64 * GROUPS * p;
            const float m1 = meet[0][other], top = fmaxf(m, m1);  // the first part has met the first key: not -inf
            const float f0 = __builtin_amdgcn_exp2f((m - top) * c), f1 = __builtin_amdgcn_exp2f((m1 - top) * c);
            add_tiles<DP / 32>(acc, f0, team.slot(tiles_, p - 1) + l, f1);
            sum = sum * f0 + meet[1][other] * f1;
            m = top;
        }
    }
    store_rows<DP>(mine, o + head * a.D, res ? res + head * a.D : nullptr, ldo, row0, at.end, a.D, acc, 1.0f / sum);
    if (h == 0 && row < at.end) lse[(int64_t)head * a.T + row] = m * a.scale + logf(sum);
    if (ordered)
        add_not_finite<false, false>(o + head * a.D, ldo, row0, min(row0 + 32, at.end), vh, a.ldv, 1,
                                     at.first - (at.first - at.begin) % kStep, a.D);
}

// dq, and the rows' statistics for the dk, dv kernel.
template <int DP, int PARTS, int GROUPS>
__global__ __launch_bounds__(64 * PARTS * GROUPS, 2) void attention_dq_kernel(
    AttentionShape a, const uint16_t *__restrict__ q, const uint16_t *__restrict__ k, const uint16_t *__restrict__ v,
    const uint16_t *__restrict__ o, const uint16_t *__restrict__ res, const float *__restrict__ lse,
    const uint16_t *__restrict__ dout, const int32_t *__restrict__ cu, uint16_t *__restrict__ dq, int64_t lddq,
    float *__restrict__ stats, int slots) {
    constexpr int OWN = 32 * GROUPS, kShare = PARTS == 1 ? 64 : 32, kStep = kShare * PARTS;
    __shared__ __attribute__((aligned(256))) uint16_t tiles_[4][kStep * DP];
    uint16_t(*ks_)[kStep * DP] = tiles_, (*vs_)[kStep * DP] = tiles_ + 2;
    __shared__ int odd;  // a result is not finite
    const int head = head_of(blockIdx.x % a.H, a.H, a.Hk), kv = head / (a.H / a.Hk);
    const Place at = place_of<OWN>(cu, a.S, a.T, slots - 1 - (int)(blockIdx.x / a.H));
    if (at.first >= at.end) return;
    const int64_t ldo = (int64_t)a.H * a.D;
    const int last = at.first + OWN < at.end ? at.first + OWN : at.end;
    if (at.outside) {
        zero_rows<OWN>(dq + head * a.D, lddq, at.first, last, a.D);
        return;
    }
    const Team<DP, PARTS, GROUPS> team;
    const int l = team.lane, h = l >> 5, part = team.part, row0 = at.first + 32 * team.group, row = row0 + (l & 31);
    Mover<DP, kStep, PARTS * GROUPS, true> mk, mv;
    mk.init(a.ldk, a.D);
    mv.init(a.ldv, a.D);
    Reader<DP, true> rd;
    rd.init(kShare * part);
    const uint16_t *kh = k + (int64_t)kv * a.D, *vh = v + (int64_t)kv * a.D;
    const int tiles = (last - at.begin + kStep - 1) / kStep;
    auto load = [&](int tile0, int b) {
        mk.load(kh, a.ldk, a.D, tile0, at.end, lds_addr(ks_[b]));
        mv.load(vh, a.ldv, a.D, tile0, at.end, lds_addr(vs_[b]));
    };
    if (threadIdx.x == 0) odd = 0;
    load(at.begin, 0);
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
    dl = -dl;
    const float ls = row < at.end ? -lse[(int64_t)head * a.T + row] / a.scale : 0.0f;
    if (part == 0 && h == 0 && row < at.end) {  // the same starting values for the dk, dv kernel
        stats[(int64_t)head * a.T + row] = ls;
        stats[(int64_t)(a.H + head) * a.T + row] = dl;
    }
    f32x16 acc[DP / 32];
    const float c = a.scale * kLog2e;
    auto start = [&] {
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[dt][i] = 0.0f;
    };
    // kc_: the keys' tile that ds is multiplied with
    auto products = [&](int tile0, const uint32_t kt_, const uint32_t vt_, const uint32_t kc_) __attribute__((always_inline)) {
        const int key0 = tile0 + kShare * part;
#pragma unroll
        for (int t = 0; t < kShare / 32; ++t) {
            const int k0 = key0 + 32 * t;
            if (k0 > row0 + 31) break;
            f32x16 s, dp;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[i] = ls;
                dp[i] = dl;
            }
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) {
                s = mfma(rd.rows(kt_, t, ks), qf[ks], s);
                dp = mfma(rd.rows(vt_, t, ks), df[ks], dp);
            }
            if (k0 + 31 > row0) {  // a branch: most tiles have nothing to mask
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (k0 + tile_row(i) > row - 4 * h) {
                        s[i] = -INFINITY;
                        dp[i] = 0.0f;
                    }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(s[i] * c) * dp[i];
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                const bf16x8 ds = operand_of(s, st);
#pragma unroll
                for (int dt = 0; dt < DP / 32; ++dt) acc[dt] = mfma(rd.cols(kc_, dt, 2 * t + st), ds, acc[dt]);
            }
        }
    };
    auto tile_step = [&](int j, auto buf) {
        constexpr int B = decltype(buf)::value;
        tile_barrier();
        const int tile0 = at.begin + j * kStep;
        if (j + 1 < tiles) load(tile0 + kStep, 1 - B);
        products(tile0, lds_addr(ks_[B]), lds_addr(vs_[B]), lds_addr(ks_[B]));
    };
    start();
    for (int j = 0; j < tiles; j += 2) {
        tile_step(j, std::integral_constant<int, 0>());
        if (j + 1 < tiles) tile_step(j + 1, std::integral_constant<int, 1>());
    }
    if (not_finite<DP / 32>(acc)) odd = 1;
    tile_barrier();  // the tiles are read
    const bool ordered = odd;
    if (ordered) {
        start();
#pragma unroll 1
        for (int j = 0; j < tiles; ++j) {
            const int tile0 = at.begin + j * kStep;
            load(tile0, 0);
            tile_barrier();
            copy_tile<kStep * DP>(lds_addr(ks_[1]), lds_addr(ks_[0]), tile0 + kStep > at.first);
            __syncthreads();
            products(tile0, lds_addr(ks_[0]), lds_addr(vs_[0]), lds_addr(ks_[1]));
            __syncthreads();
        }
    }
    float *mine = team.slot(tiles_, 0);
    if (PARTS > 1) {
        if (part > 0) put_tiles<DP / 32>(team.slot(tiles_, part - 1) + l, acc);
        __syncthreads();
        if (part > 0) return;
#pragma unroll
        for (int p = 1; p < PARTS; ++p) add_tiles<DP / 32>(acc, 1.0f, team.slot(tiles_, p - 1) + l, 1.0f);
    }
    store_rows<DP>(mine, dq + head * a.D, nullptr, lddq, row0, at.end, a.D, acc, a.scale);
    if (ordered)
        add_not_finite<false, true>(dq + head * a.D, lddq, row0, min(row0 + 32, at.end), kh, a.ldk, 1,
                                    at.first - (at.first - at.begin) % kStep, a.D);
}

// Where the dk, dv kernel's results go: the gradients, or with `part` one fp32
// partial a head ([2][H][T][D]: dk, dv) for the kernel that adds a group's heads.
struct KvOut {
    uint16_t *dk, *dv;
    int64_t lddk, lddv;
    float *part;
};

// Stores a transposed result times f as fp32 rows.
template <int DP>
__device__ __forceinline__ void store_rows_f32(float *y, int64_t ld, int row0, int end, int D, const f32x16 *t, float f) {
    const int l = threadIdx.x & 63, h = l >> 5, row = row0 + (l & 31);
    if (row >= end) return;
#pragma unroll
    for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const int c = 32 * dt + tile_row(i) + 4 * h;
            if (c < D)
                *reinterpret_cast<f32x4 *>(y + (int64_t)row * ld + c) =
                    f32x4{t[dt][i] * f, t[dt][i + 1] * f, t[dt][i + 2] * f, t[dt][i + 3] * f};
        }
}

// dk and dv of OWN keys: all rows from them on, of one head (SPLIT: a workgroup a
// head, partial results) or of all heads of the group.  The keys stay in LDS and
// the values in registers: with both in registers the two accumulators leave no
// room for two waves a SIMD.
template <int DP, bool SPLIT, int PARTS, int GROUPS>
__global__ __launch_bounds__(64 * PARTS * GROUPS, 2) void attention_dkv_kernel(
    AttentionShape a, const uint16_t *__restrict__ q, const uint16_t *__restrict__ k, const uint16_t *__restrict__ v,
    const float *__restrict__ stats, const uint16_t *__restrict__ dout, const int32_t *__restrict__ cu, KvOut out) {
    constexpr int OWN = 32 * GROUPS, kTile = 32 * PARTS;
    __shared__ __attribute__((aligned(256))) uint16_t lds_[(OWN + 4 * kTile) * DP];
    uint16_t *ks_ = lds_;
    uint16_t(*qs_)[kTile * DP] = reinterpret_cast<uint16_t(*)[kTile * DP]>(lds_ + OWN * DP), (*ds_)[kTile * DP] = qs_ + 2;
    static_assert(PARTS == 1 || (PARTS - 1) * GROUPS * DP / 2 * 64 * 4 <= sizeof(lds_), "the parts' results");
    __shared__ __attribute__((aligned(16))) float ls_[2][kTile], dl_[2][kTile];
    __shared__ int odd;  // a result is not finite
    const int group = a.H / a.Hk, heads = SPLIT ? a.H : a.Hk;
    const int first_head = SPLIT ? head_of(blockIdx.x % a.H, a.H, a.Hk) : (int)(blockIdx.x % a.Hk) * group;
    const int kv = first_head / group;
    const Place at = place_of<OWN>(cu, a.S, a.T, (int)(blockIdx.x / heads));  // the first keys have the most rows
    if (at.first >= at.end) return;
    const int64_t ldo = (int64_t)a.H * a.D;
    float *pk = SPLIT ? out.part + (int64_t)first_head * a.T * a.D : nullptr;
    float *pv = SPLIT ? out.part + ((int64_t)a.H + first_head) * a.T * a.D : nullptr;
    if (at.outside) {
        const int last = at.first + OWN < at.end ? at.first + OWN : at.end;
        if (SPLIT) {
            zero_rows<OWN>(reinterpret_cast<uint16_t *>(pk), 2 * a.D, at.first, last, 2 * a.D);
            zero_rows<OWN>(reinterpret_cast<uint16_t *>(pv), 2 * a.D, at.first, last, 2 * a.D);
        } else {
            zero_rows<OWN>(out.dk + kv * a.D, out.lddk, at.first, last, a.D);
            zero_rows<OWN>(out.dv + kv * a.D, out.lddv, at.first, last, a.D);
        }
        return;
    }
    const Team<DP, PARTS, GROUPS> team;
    const int l = team.lane, h = l >> 5, part = team.part, key0 = at.first + 32 * team.group, key = key0 + (l & 31);
    Mover<DP, kTile, PARTS * GROUPS, true> mq, md;
    mq.init(a.ldq, a.D);
    md.init(ldo, a.D);
    Reader<DP, true> rd;
    rd.init(32 * part);
    // A tile of rows and their statistics.  Rows past the end are zeros throughout: p = 1
    // there, against do = 0 and q = 0.
    auto fetch = [&](int hd, int r0, int b) {
        mq.load(q + (int64_t)hd * a.D, a.ldq, a.D, r0, at.end, lds_addr(qs_[b]));
        md.load(dout + (int64_t)hd * a.D, ldo, a.D, r0, at.end, lds_addr(ds_[b]));
        constexpr int kPieces = (kTile + 63) / 64;  // of 64 statistics
        if (team.wave < 2 * kPieces && l < kTile) {
            const int which = team.wave & 1, from = (team.wave >> 1) * 64;
            const __amdgpu_buffer_rsrc_t r =
                out_rsrc(stats + (int64_t)(which * a.H + hd) * a.T + r0, (int64_t)(at.end - r0) * 4);
            transfer4(r, lds_addr((which ? dl_[b] : ls_[b]) + from), (from + l) * 4);
        }
    };
    int hd = first_head, r0 = at.first;  // of the tile at hand
    {
        Mover<DP, OWN, PARTS * GROUPS, false> mk;
        mk.init(a.ldk, a.D);
        mk.load(k + (int64_t)kv * a.D, a.ldk, a.D, at.first, at.end, lds_addr(ks_));
    }
    if (threadIdx.x == 0) odd = 0;
    fetch(hd, r0, 0);
    bf16x8 vf[DP / 16];
    load_rows<DP>(v + (int64_t)kv * a.D, a.ldv, key0, at.end, a.D, vf);
    f32x16 ak[DP / 32], av[DP / 32];
    auto start = [&] {
#pragma unroll
        for (int dt = 0; dt < DP / 32; ++dt)
#pragma unroll
            for (int i = 0; i < 16; ++i) ak[dt][i] = av[dt][i] = 0.0f;
    };
    const float c = a.scale * kLog2e;
    uint32_t kt_ = lds_addr(ks_) + 32 * (team.group - part) * DP * 2;  // the reader is 32 part rows ahead
    const int per = (at.end - at.first + kTile - 1) / kTile, tiles = per * (SPLIT ? 1 : group);
    // The tile of rows from r0 on, in buffer B; C: the one whose columns p and ds are multiplied with
    auto products = [&](int r0, auto buf, auto cols) __attribute__((always_inline)) {
        constexpr int B = decltype(buf)::value, C = decltype(cols)::value;
        const uint32_t qt_ = lds_addr(qs_[B]), dt_ = lds_addr(ds_[B]), qc_ = lds_addr(qs_[C]), dc_ = lds_addr(ds_[C]);
        const uint32_t lt_ = lds_addr(ls_[B]) + 16 * h + 128 * part, et_ = lds_addr(dl_[B]) + 16 * h + 128 * part;
        const int q0 = r0 + 32 * part;
        if (q0 + 31 < key0) return;  // these rows all come before the wave's keys
        asm volatile("" : "+s"(kt_));  // read the keys again, do not keep their fragments over the loop
        f32x16 s, dp;
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const f32x4 ls = *reinterpret_cast<const lds_f32x4 *>(lt_ + 2 * i * 4);
            const f32x4 dl = *reinterpret_cast<const lds_f32x4 *>(et_ + 2 * i * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[i + e] = ls[e];
                dp[i + e] = dl[e];
            }
        }
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) {
            s = mfma(rd.rows(qt_, 0, ks), rd.rows(kt_, 0, ks), s);
            dp = mfma(rd.rows(dt_, 0, ks), vf[ks], dp);
        }
        if (q0 < key0 + 31) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (q0 + tile_row(i) < key - 4 * h) {
                    s[i] = -INFINITY;
                    dp[i] = 0.0f;
                }
        }
        u32x4 pw[2], sw[2];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float p0 = __builtin_amdgcn_exp2f(s[i] * c), p1 = __builtin_amdgcn_exp2f(s[i + 1] * c);
            pw[i / 8][i / 2 % 4] = pack_bf16x2(p0, p1);
            sw[i / 8][i / 2 % 4] = pack_bf16x2(p0 * dp[i], p1 * dp[i + 1]);
        }
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const bf16x8 pb = __builtin_bit_cast(bf16x8, pw[st]), sb = __builtin_bit_cast(bf16x8, sw[st]);
#pragma unroll
            for (int dt = 0; dt < DP / 32; ++dt) {
                av[dt] = mfma(rd.cols(dc_, dt, st), pb, av[dt]);
                ak[dt] = mfma(rd.cols(qc_, dt, st), sb, ak[dt]);
            }
        }
    };
    typedef std::integral_constant<int, 0> Zero;
    typedef std::integral_constant<int, 1> One;
    auto next_tile = [&] {
        r0 += kTile;
        if (r0 >= at.end) {
            ++hd;
            r0 = at.first;
        }
    };
    auto tile_step = [&](int j, auto buf) {
        constexpr int B = decltype(buf)::value;
        tile_barrier();
        const int now = r0;
        next_tile();
        if (j + 1 < tiles) fetch(hd, r0, 1 - B);
        products(now, buf, buf);
    };
    start();
    for (int j = 0; j < tiles; j += 2) {
        tile_step(j, Zero());
        if (j + 1 < tiles) tile_step(j + 1, One());
    }
    if (not_finite<DP / 32>(ak) || not_finite<DP / 32>(av)) odd = 1;
    tile_barrier();  // the tiles are read
    const bool ordered = odd;
    if (ordered) {
        start();
        hd = first_head;
        r0 = at.first;
#pragma unroll 1
        for (int j = 0; j < tiles; ++j, next_tile()) {
            fetch(hd, r0, 0);
            tile_barrier();
            copy_tile<kTile * DP>(lds_addr(qs_[1]), lds_addr(qs_[0]), r0 < at.first + OWN);
            copy_tile<kTile * DP>(lds_addr(ds_[1]), lds_addr(ds_[0]), r0 < at.first + OWN);
            __syncthreads();
            products(r0, Zero(), One());
            __syncthreads();
        }
    }
    // dk is the first part's to add and store, dv the second's, one after the other
    float *mine = team.slot(lds_, 0);
    if (PARTS > 1) {
        if (part > 0) put_tiles<DP / 32>(team.slot(lds_, part - 1) + l, ak);
        __syncthreads();
    }
    if (part == 0) {
#pragma unroll 1
        for (int p = 1; p < PARTS; ++p) add_tiles<DP / 32>(ak, 1.0f, team.slot(lds_, p - 1) + l, 1.0f);
        if (SPLIT) store_rows_f32<DP>(pk, a.D, key0, at.end, a.D, ak, a.scale);
        else store_rows<DP>(mine, out.dk + kv * a.D, nullptr, out.lddk, key0, at.end, a.D, ak, a.scale);
    }
    if (PARTS > 1) {
        __syncthreads();
        if (part != 1) put_tiles<DP / 32>(team.slot(lds_, part > 1 ? part - 1 : 0) + l, av);
        __syncthreads();
    }
    if (part == (PARTS > 1 ? 1 : 0)) {
#pragma unroll 1
        for (int p = 1; p < PARTS; ++p) add_tiles<DP / 32>(av, 1.0f, team.slot(lds_, p - 1) + l, 1.0f);
        if (SPLIT) store_rows_f32<DP>(pv, a.D, key0, at.end, a.D, av, 1.0f);
        else store_rows<DP>(mine, out.dv + kv * a.D, nullptr, out.lddv, key0, at.end, a.D, av, 1.0f);
        if (ordered) {  // (dk has them: a row whose q, k, v or do is not finite has no finite ds)
            const uint16_t *dh = dout + (int64_t)first_head * a.D;
            const int end = min(key0 + 32, at.end), start = min(at.first + (OWN > kTile ? OWN : kTile), at.end);
            if (SPLIT) add_not_finite<true, false>(pv, a.D, key0, end, dh, ldo, 1, start, a.D);
            else add_not_finite<true, false>(out.dv + kv * a.D, out.lddv, key0, end, dh, ldo, group, start, a.D);
        }
    }
}

// dk (blockIdx.y 0) and dv (1) from the heads' partials, added in head order.
__global__ __launch_bounds__(kThreads) void attention_group_sum_kernel(AttentionShape a, KvOut out) {
    const int chunks = a.D / 8;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, n = (int64_t)a.T * a.Hk * chunks;
    if (i >= n) return;
    const int64_t row = i / (a.Hk * chunks);
    const int kv = (int)(i / chunks % a.Hk), c = (int)(i % chunks) * 8, group = a.H / a.Hk;
    const float *p = out.part + (((int64_t)blockIdx.y * a.H + kv * group) * a.T + row) * a.D + c;
    f32x4 lo = {}, hi = {};
    for (int g = 0; g < group; ++g, p += (int64_t)a.T * a.D) {
        lo += *reinterpret_cast<const f32x4 *>(p);
        hi += *reinterpret_cast<const f32x4 *>(p + 4);
    }
    uint16_t *y = (blockIdx.y ? out.dv + row * out.lddv : out.dk + row * out.lddk) + kv * a.D + c;
    *reinterpret_cast<uint4 *>(y) = make_uint4(pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]),
                                               pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3]));
}

// Slots of a head for workgroups of `own` rows.
int slots_of(const AttentionShape &a, int own) { return a.T / own + a.S + 2; }

// A workgroup a head instead of a group in the dk, dv kernel.  With a group a
// workgroup, the first keys of a sequence of L rows take group L / 32 steps, and the
// launch no less; shared evenly over the 512 resident workgroups, all of them would
// take T H L / 2^22.  The partials cost 16 T H D bytes of traffic, as much as about
// T H / 2700 steps, and half of the uneven rest is won back (workgroups alone on a
// CU run faster).  L is the mean length T / S: the lengths are on the device.  Backward
// in all (us, a head / a group a workgroup), D = 128, H / Hk = 32 / 8: 4 x 1024 228 / 266, 4 x 2048 590 / 640,
// 1 x 8192 1805 / 2315; 8 x 1024 408 / 353, 16 x 512 329 / 238, 16 x 1024 783 / 674.
bool split_heads(const AttentionShape &a) {
    const double len = a.T / a.S;
    return a.H > a.Hk && len * 131072 > (double)a.T * a.Hk * (len + 1536);
}

// Parts, from the mean length L of the sequences (the lengths themselves are on the
// device) and the T H rows of all heads, which make T H / 64 workgroups of four parts.
// Four where these run in one round: LDS leaves one a CU for D > 64, registers one in the
// backward (150 to 160: three waves a SIMD, a workgroup takes two); forward for D <= 64 two.
// Or where one long sequence is most of it.  Forward + backward, one part / two / four (us):
// 1 x 1024 H / Hk 8 / 8 D 128 94 / 82 / 64, 2 x 512 16 / 16 D 128 60 / 58 / 50, (1000, 20, 20, 20, 20) 8 / 4 D 64
// 69 / 58 / 43, 4 x 256 8 / 8 D 128 40 / 43 / 40; beyond: 3 x 512 16 / 16 D 128 63 / 60 / 83, 8 x 128 16 / 4 D 128
// 45 / 51 / 52.  D = 64, T H from 16384 to 32768, forward alone: (700, 3, 517, 1, 250, 1025) 12 / 4 20 / 19 / 16,
// 1 x 2048 16 / 4 31 / 25 / 20, 4 x 512 12 / 12 11.7 / 10.8 / 12.2, 6 x 300 14 / 14 9.4 / 10.7 / 11.2 (what equal
// lengths lose is less than what others gain); backward alone, T H up to 32 L: 1 x 1024 20 / 20 48 / 41 / 34,
// 1 x 2048 16 / 4 94 / 74 / 64, 1 x 768 32 / 32 39 / 34 / 34; beyond: 4 x 512 12 / 12 31 / 29 / 36, 6 x 300 14 / 14
// 25 / 24 / 35, 8 x 256 16 / 16 24 / 24 / 34, the batch of 12 / 4 58 / 52 / 51, (3000, 9 times 20) 9 / 3 126 / 95 / 76.
// Two, of 128 rows, where the workgroups are no more than the 512 that run at a time
// with one part: 1 x 8192 8 / 2 D 128 812 / 645, 2 x 2048 16 / 16 D 64 174 / 137, (2570, 37, 34, 0, 110, 2, 14, 5)
// 8 / 8 D 128 204 / 169; beyond: 4 x 512 32 / 32 D 64 67 / 75, 1 x 8192 16 / 4 D 128 1228 / 1267.  Shorter sequences
// where a backward's are one a CU: D 64 8 x 210 14 / 14 25 / 21, 8 x 256 12 / 4 36 / 31, 7 x 280 14 / 14 30 / 35.
int parts_of(const AttentionShape &a, bool backward) {
    const int64_t len = a.T / a.S, rows = (int64_t)a.T * a.H;
    const bool narrow = a.D <= 64, half = rows <= 32768;
    const bool one_round = rows <= 16384 || (narrow && !backward && half);
    if (len >= 200 && (one_round || (half && rows <= (narrow ? 32 : 12) * len))) return 4;
    if (len >= 200 && narrow && backward && half) return 2;
    return len >= 300 && rows <= 65536 && rows <= 80 * len ? 2 : 1;
}
size_t stats_bytes(const AttentionShape &a) { return (sizeof(float) * 2 * (size_t)a.T * a.H + 255) / 256 * 256; }

template <int DP, int PARTS, int GROUPS>
hipError_t backward(const AttentionShape &a, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                    const uint16_t *o, const uint16_t *res, const float *lse, const uint16_t *dout, const int32_t *cu,
                    uint16_t *dq, int64_t lddq, float *stats, const KvOut &out, hipStream_t s) {
    constexpr int kT = 64 * PARTS * GROUPS;
    const int slots = slots_of(a, 32 * GROUPS);
    attention_dq_kernel<DP, PARTS, GROUPS>
        <<<(unsigned)slots * a.H, kT, 0, s>>>(a, q, k, v, o, res, lse, dout, cu, dq, lddq, stats, slots);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (!split_heads(a)) {
        attention_dkv_kernel<DP, false, PARTS, GROUPS><<<(unsigned)slots * a.Hk, kT, 0, s>>>(a, q, k, v, stats, dout, cu, out);
        return hipGetLastError();
    }
    attention_dkv_kernel<DP, true, PARTS, GROUPS><<<(unsigned)slots * a.H, kT, 0, s>>>(a, q, k, v, stats, dout, cu, out);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t chunks = (int64_t)a.T * a.Hk * (a.D / 8);
    attention_group_sum_kernel<<<dim3((unsigned)((chunks + kThreads - 1) / kThreads), 2), kThreads, 0, s>>>(a, out);
    return hipGetLastError();
}

// f with the padded head dimension, the parts and the groups as template values.
template <typename F>
hipError_t shaped(const AttentionShape &a, bool backward, F f) {
    auto with = [&](auto dp) {
        switch (parts_of(a, backward)) {
            case 4: return f(dp, std::integral_constant<int, 4>(), std::integral_constant<int, 2>());
            case 2: return f(dp, std::integral_constant<int, 2>(), std::integral_constant<int, 4>());
            default: return f(dp, std::integral_constant<int, 1>(), std::integral_constant<int, 4>());
        }
    };
    return a.D <= 64 ? with(std::integral_constant<int, 64>()) : with(std::integral_constant<int, 128>());
}

}  // namespace

int64_t attention_groups(const AttentionShape &a) { return (int64_t)slots_of(a, 64) * a.H; }

size_t attention_bwd_bytes(const AttentionShape &a) {
    return stats_bytes(a) + (split_heads(a) ? sizeof(float) * 2 * (size_t)a.T * a.H * a.D : 0);
}

hipError_t launch_attention_fwd(const AttentionShape &a, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                                const int32_t *cu, uint16_t *o, uint16_t *res, float *lse, hipStream_t s) {
    return shaped(a, false, [&](auto dp, auto parts, auto groups) {
        constexpr int kDp = decltype(dp)::value, kParts = decltype(parts)::value, kGroups = decltype(groups)::value;
        const int slots = slots_of(a, 32 * kGroups);
        attention_fwd_kernel<kDp, kParts, kGroups>
            <<<(unsigned)slots * a.H, 64 * kParts * kGroups, 0, s>>>(a, q, k, v, cu, o, res, lse, slots);
        return hipGetLastError();
    });
}

hipError_t launch_attention_bwd(const AttentionShape &a, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                                const uint16_t *o, const uint16_t *res, const float *lse, const uint16_t *dout,
                                const int32_t *cu, uint16_t *dq, int64_t lddq, uint16_t *dk, int64_t lddk,
                                uint16_t *dv, int64_t lddv, void *ws, hipStream_t s) {
    float *stats = static_cast<float *>(ws);
    const KvOut out{dk, dv, lddk, lddv, reinterpret_cast<float *>(static_cast<char *>(ws) + stats_bytes(a))};
    return shaped(a, true, [&](auto dp, auto parts, auto groups) {
        return backward<decltype(dp)::value, decltype(parts)::value, decltype(groups)::value>(a, q, k, v, o, res, lse, dout, cu, dq, lddq, stats, out, s);
    });
}

}  // namespace qnf4
