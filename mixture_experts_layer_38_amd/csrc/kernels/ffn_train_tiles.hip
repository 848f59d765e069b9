// The grouped products of the expert FFN in training, in bf16 (formulas:
// ffn_train.hip).  Most have operands that are contiguous across the reduction:
//   TR_DACT  da = dh W2_e                 rows [r][k] times [k][n]; epilogue: dgate, dup, act
//   TR_DX    dx = dgate W1_e + dup W3_e   two such products into one sum
//   TR_DW    dW = P^T Q                   [r][m] times [r][n], the sum over the expert's rows
// and for widths that the forward pass's tiled kernel does not take (no
// multiples of 64)
//   TR_GATE  gate, up = rows [r][k] times W1_e, W3_e [n][k]; epilogue: act as well
//   TR_DOWN  h = act W2_e^T               the same with one weight
//
// Tiles of BM x 256 outputs on four waves (2 x 2), v_mfma_f32_32x32x16_bf16
// with the n side as the first operand, so a lane ends with four consecutive
// outputs of a row; fp32 accumulators fill the AGPRs.
//
// A stage is 64 wide in k.  A [k][n] operand lies in the LDS as 64 rows of 512
// bytes and its fragments come from ds_read_b64_tr_b16, which hands each lane
// of 16 one column of a 4 x 16 block: lane 4 r + c addresses elements
// 4 c .. 4 c + 3 of row r, and lane i gets column i of the four rows.  Two such
// reads give the eight k of a lane.  The 16-byte chunk c of row k is kept in
// slot c ^ 4 (k % 4), so the 32-byte pieces of the four rows of both 16-lane
// groups lie in distinct banks.  A [r][k] operand lies in 128-byte rows as in
// the forward kernel (pf_swz).
//
// Stages go straight into the LDS with buffer loads: the descriptor carries
// the stage's address and how many bytes of it exist, so rows past the end of
// the group, of the reduction or of the matrix arrive as zeros and nothing
// past an operand's last element is ever read.
//
// Bounds.  Long groups: the matrix pipes, at the clock that power allows
// (16384 rows, 8 experts, d 4096, F 14336: da 1.77 ms, the three weight gradients
// 4.54, dx 3.28, together 9.6 ms, 1200 TFLOP/s; a large library product reaches
// 1210).  Short groups: the weights' bytes (4096 rows, 32 experts, d 7168, F
// 2048: da 187 us and dx 437 us at 5.0 and 4.3 TB/s; the weight gradients 770 to
// 850 us, 3.5 TB/s of writes: with one stage of rows the same tiles are written at 6
// TB/s, so what is left there is the operands' way into the LDS, which the
// stores of the other workgroup of the CU hide only in part).  The weight
// gradients share a launch, and row tiles of up to 64 experts are found without
// a plan launch, for small layers (333 tokens, 5 experts, K 3, d 264, F 200: 45
// -> 34 us; the large ones above stay within the noise).
#include <algorithm>
#include <type_traits>

#include "../device_common.h"
#include "../launch.h"
#include "ffn_tiles.h"
#include "gated.h"

namespace moe {

namespace {

enum { TR_DACT, TR_DX, TR_DW, TR_GATE, TR_DOWN };
constexpr int TR_BN = 256;
// Rows per expert from which TR_DW takes 256 x 256 tiles, one workgroup per CU;
// shorter groups take 128 x 256, two per CU, since a tile's loads and its stores
// then overlap (dW1 and dW3 of the 128 rows per expert above: 634 -> 570 us).
constexpr int TR_DW_LONG = 512;
constexpr int TR_GM = 8;  // row tiles per group in TR_DW's order

struct TrainArgs {
    const bf16 *a0, *a1, *a2;  // rows (TR_DX: of both products; TR_DW: the m sides of its three results)
    const bf16 *b0, *b1, *b2;  // the n side (TR_GATE: both weights; TR_DW: of the three results)
    bf16 *out0, *out1, *out2;
    const bf16 *gate, *up;
    int n_rows, E;
    // [rows][N], K the reduction of one product; TR_DW: an expert's first result
    // is [M][N], the other two [N][M]
    int M, N, K;
    int lda, ldb, n_nt;
    // Ranges of the reduction that are summed apart when there are several:
    // TR_DW, of rows, into part [parts][E][3][M N]; TR_DX and TR_DOWN, of
    // stages, into part [parts][rows][N].
    int parts;
    float* part;
    RowPlan plan;  // mt_count NULL: up to 64 experts, whose row tiles each workgroup finds itself
    const int32_t* offsets;
};

// KT: K is not a multiple of the stage, so a [r][k] row's chunks past it are
// masked (they would be the next row's; TR_DW has no such rows).
// PART: fp32 sums of one range of the reduction.
template <int MODE, int BM, bool KT, bool PART = false>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(BM == 256 ? 1 : 2, BM == 256 ? 1 : 2)))
void ffn_train_kernel(TrainArgs g) {
    constexpr bool WG = MODE == TR_DW;
    constexpr bool BROWS = MODE == TR_GATE || MODE == TR_DOWN;  // the n side lies in [n][k] rows
    constexpr int TR_BK = BM == 256 ? 64 : 32;  // k per stage
    constexpr int SA = BM * TR_BK, SB = TR_BN * TR_BK;  // elements of a stage's halves
    constexpr int NTB = BM / 64;   // 32-wide m blocks per wave
    constexpr int NJA = SA / 2048, NJB = SB / 2048, NLD = NJA + NJB;  // loads per wave and stage
    constexpr bool RING5 = BM == 256;
    // BM 256: five 32 KB units that the halves of consecutive stages take in
    // turn; BM 128: three slots of 24 KB for whole stages (two workgroups per CU).
    __shared__ __align__(1024) bf16 sA0[SA], sA1[SA], sA2[RING5 ? 1 : SA];
    __shared__ __align__(1024) bf16 sB0[SB], sB1[SB], sB2[RING5 ? 1 : SB];
    __shared__ __align__(1024) bf16 sU4[RING5 ? SB : 1];

    const int xcd = blockIdx.x % PF_XCD, slot = blockIdx.x / PF_XCD;
    int e, row0 = 0, row_end = 0, m0 = 0, n0, k_beg = 0, k_len = g.K;
    int range = 0;  // of g.parts
    const bf16 *A0 = g.a0, *A1 = g.a1, *B0 = g.b0, *B1 = g.b1;
    bf16* out = g.out0;
    int M = g.M, N = g.N, lda = g.lda, ldb = g.ldb;
    int sel = 0;  // TR_DW: which of the expert's results
    // Uniform values are put into scalar registers (divisions and lane reads run
    // in vector ones), so that the descriptors made of them are scalar too.
    const auto uni = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    if constexpr (WG) {
        // every XCD takes an eighth of each result's tiles: the experts' row
        // counts differ, the XCDs' shares of them do not
        const auto tiles_of = [](int m, int n) { return ((m + BM - 1) / BM) * ((n + TR_BN - 1) / TR_BN); };
        const int per0 = (tiles_of(M, N) + PF_XCD - 1) / PF_XCD, per1 = (tiles_of(N, M) + PF_XCD - 1) / PF_XCD;
        const int per_e = (per0 + 2 * per1) * g.parts;
        e = uni(slot / per_e);
        if (e >= g.E) return;
        int r = uni(slot - e * per_e), per = per0;
        if (r >= per0 * g.parts) {
            r -= per0 * g.parts;
            per = per1;
            sel = uni(1 + r / (per1 * g.parts));
            r = uni(r % (per1 * g.parts));
            M = lda = g.N;
            N = ldb = g.M;
            A0 = sel == 1 ? g.a1 : g.a2;
            B0 = sel == 1 ? g.b1 : g.b2;
            out = sel == 1 ? g.out1 : g.out2;
        }
        range = uni(r / per);
        const int t = xcd * per + uni(r % per);
        if (t >= tiles_of(M, N)) return;
        const int n_mt = (M + BM - 1) / BM, n_nt = (N + TR_BN - 1) / TR_BN;
        const int grp = t / (TR_GM * n_nt), gsize = min(TR_GM, n_mt - grp * TR_GM);
        const int rem = t - grp * TR_GM * n_nt;
        m0 = uni((grp * TR_GM + rem % gsize) * BM);
        n0 = uni(rem / gsize * TR_BN);
        k_beg = uni(min(max(g.offsets[e], 0), g.n_rows));
        k_len = max(uni(min(g.offsets[e + 1], g.n_rows)) - k_beg, 0);
        out += (size_t)e * M * N;
        if constexpr (PART) {  // whole stages, but for the last range's end
            const int beg = (int)((long long)k_len * range / g.parts) & ~63;
            const int end = range + 1 < g.parts ? (int)((long long)k_len * (range + 1) / g.parts) & ~63 : k_len;
            k_beg += beg;
            k_len = end - beg;
        } else if (k_len == 0) {  // an expert without rows: zeros, by whole lines
            const int c = n0 + (threadIdx.x & 31) * 8;
            for (int r = m0 + threadIdx.x / 32; r < min(m0 + BM, M); r += 8)
                if (c < N) *reinterpret_cast<u32x4*>(out + (size_t)r * N + c) = u32x4{0, 0, 0, 0};
            return;
        }
    } else {
        const GroupTiles gt(g.plan, g.E, BM, g.offsets);
        const int tiles = gt.count * g.n_nt;
        const int per = (tiles * (PART ? g.parts : 1) + PF_XCD - 1) / PF_XCD;
        int t = xcd * per + slot;
        if (slot >= per || t >= tiles * (PART ? g.parts : 1)) return;
        if constexpr (PART) {
            range = uni(t % g.parts);
            t /= g.parts;
        }
        const PfTile tl = gt.tile(t, g.n_nt, g.n_rows);
        e = uni(tl.e);
        row0 = uni(tl.row0);
        row_end = min(uni(tl.row_end), row0 + BM);
        if (row0 >= row_end) return;  // (offsets past the rows)
        n0 = uni(tl.nt) * (MODE == TR_GATE ? 128 : TR_BN);
        const size_t we = (size_t)e * g.K * g.N;
        B0 += we;
        if (MODE == TR_DX || MODE == TR_GATE) B1 += we;
    }
    const int nk1 = (k_len + TR_BK - 1) / TR_BK;  // stages of one product
    const int nk_all = MODE == TR_DX ? 2 * nk1 : nk1;
    // this workgroup's stages: all, or a range of them (TR_DW's ranges are in k_beg and k_len)
    constexpr bool RANGE = PART && !WG;
    const int ks = RANGE ? nk_all * range / g.parts : 0;
    const int ke = RANGE ? nk_all * (range + 1) / g.parts : nk_all;
    const int nk = ke - ks;

    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    const int lane = lane_id();

    // ---- loads -------------------------------------------------------------------
    // [r][k] halves: instruction j of wave w fills rows 8 (w + 4 j) .. + 7 of 128
    // bytes, whose swizzle depends on j's lowest bit, or rows 16 (w + 4 j) .. + 15
    // of 64 bytes.  off[j & 1]: the lane's byte offset at j = 0 (rows `back` fewer),
    // first[j & 1]: the first k of its chunk.
    auto row_chunks = [&](int back, uint32_t (&off)[2], int (&first)[2], int ld) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (TR_BK == 32) {
                first[i] = ((lane & 3) ^ ((lane >> 3) & 3)) * 8;
                off[i] = (uint32_t)((16 * wave - back + (lane >> 2)) * ld + first[i]) * 2;
            } else {
                first[i] = ((lane & 7) ^ pf_swz(8 * (wave + 4 * i) + (lane >> 3))) * 8;
                off[i] = (uint32_t)((8 * wave + (lane >> 3)) * ld + first[i]) * 2;
            }
        }
    };
    // [k][n] halves: instruction j of wave w fills rows 2 (w + 4 j) and the next
    // ([k][m] with 128 m: four rows from 4 (w + 4 j)); lane p slot p % 32 (16).
    const int brow = 2 * wave + (lane >> 5);
    uint32_t vb[2] = {(uint32_t)(brow * ldb + ((lane & 31) ^ ((brow & 3) << 2)) * 8) * 2, 0};
    constexpr int ACH = BM / 8;           // chunks of a [k][m] row
    constexpr int ARI = kWave / ACH;      // rows of one instruction
    uint32_t va[2];
    int ac[2];
    if constexpr (WG) {
        const int arow = ARI * wave + lane / ACH;
        va[0] = va[1] = (uint32_t)(arow * lda + ((lane % ACH) ^ ((arow & 3) << 2)) * 8) * 2;
        ac[0] = ac[1] = 0;
    } else {
        row_chunks(0, va, ac, lda);
    }
    // [n][k] halves: as [r][k] ones, of 256 weight rows.  TR_GATE: 128 rows of
    // each weight in alternating blocks of 32, so a lane's gate and up sums meet;
    // a wave instruction then fetches rows of one weight: with 64 k a stage, of
    // W1 for even j and W3 for odd, with 32, of W1 in waves 0 and 1.
    int bc[2] = {0, 0};
    if constexpr (BROWS) row_chunks(MODE == TR_GATE && TR_BK == 32 ? 16 * (wave & 2) : 0, vb, bc, ldb);
    // Descriptors of stage kt: its first element and the bytes from there on that exist.
    auto rsrc = [&](const bf16* p, int bytes) __attribute__((always_inline)) {
        return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, bytes, 0x00020000);
    };
    auto rs_a = [&](int kt) __attribute__((always_inline)) {
        if constexpr (WG) {
            const int v = min(max(k_len - kt * TR_BK, 0), TR_BK);
            return rsrc(A0 + (size_t)(k_beg + kt * TR_BK) * lda + m0, v > 0 ? (v * lda - m0) * 2 : 0);
        } else {
            const int seg = MODE == TR_DX && kt >= nk1;
            const int k0 = (kt - (seg ? nk1 : 0)) * TR_BK;
            const int bytes = kt < ke ? ((row_end - row0) * lda - k0) * 2 : 0;
            return rsrc((seg ? A1 : A0) + (size_t)row0 * lda + k0, bytes);
        }
    };
    auto rs_b = [&](int kt, int which = 0) __attribute__((always_inline)) {
        if constexpr (BROWS) {
            const int bytes = kt < ke ? (min(N - n0, MODE == TR_GATE ? 128 : TR_BN) * ldb - kt * TR_BK) * 2 : 0;
            return rsrc((which ? B1 : B0) + (size_t)n0 * ldb + kt * TR_BK, bytes);
        }
        const int seg = MODE == TR_DX && kt >= nk1;
        const int k0 = (kt - (seg ? nk1 : 0)) * TR_BK;
        const int v = kt < ke ? min(k_len - k0, TR_BK) : 0;
        return rsrc((seg ? B1 : B0) + (size_t)(k_beg + k0) * ldb + n0, v > 0 ? (v * ldb - n0) * 2 : 0);
    };
    auto ld_a = [&](__amdgpu_buffer_rsrc_t r, int kt, int j, bf16* dst) __attribute__((always_inline)) {
        uint32_t v = va[j & 1];
        if constexpr (KT && !WG) {
            const int k0 = (kt - (MODE == TR_DX && kt >= nk1 ? nk1 : 0)) * TR_BK;
            v = ac[j & 1] < k_len - k0 ? v : 0x80000000u;  // past every descriptor's bytes
        }
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            r, (__attribute__((address_space(3))) void*)(dst + (wave + 4 * j) * 512), 16, v,
            WG ? j * (4 * ARI * 2) * lda : j * (4096 / TR_BK) * lda, 0, 0);
    };
    auto ld_b = [&](const __amdgpu_buffer_rsrc_t (&r)[2], int kt, int j, bf16* dst) __attribute__((always_inline)) {
        uint32_t v = vb[BROWS ? j & 1 : 0];
        if constexpr (KT && BROWS) v = bc[j & 1] < k_len - kt * TR_BK ? v : 0x80000000u;
        // rows that a step of j moves on by
        constexpr int JR = !BROWS ? 8 : 4096 / TR_BK / 2 / (MODE == TR_GATE && TR_BK == 32 ? 2 : 1);
        const int rows = MODE == TR_GATE && TR_BK == 64 ? (j >> 1) * JR : j * JR;
        const int which = MODE != TR_GATE ? 0 : TR_BK == 64 ? j & 1 : 0;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            r[which], (__attribute__((address_space(3))) void*)(dst + (wave + 4 * j) * 512), 16, v, rows * 2 * ldb, 0, 0);
    };
    // The weights' descriptors of stage kt (TR_GATE with 32 k a stage: each wave's own weight).
    struct RsB {
        __amdgpu_buffer_rsrc_t r[2];
    };
    auto rs_bs = [&](int kt) __attribute__((always_inline)) {
        if constexpr (MODE == TR_GATE && TR_BK == 64) return RsB{{rs_b(kt, 0), rs_b(kt, 1)}};
        else if constexpr (MODE == TR_GATE) return RsB{{rs_b(kt, wave >> 1), rs_b(kt, wave >> 1)}};
        else return RsB{{rs_b(kt), rs_b(kt)}};
    };

    // ---- fragments ------------------------------------------------------------------
    const int wm = wave & 1, wn = wave >> 1;
    const int fhalf = lane >> 5, g16 = (lane >> 4) & 1, rr = (lane >> 2) & 3, cc = lane & 3;
    // element offsets inside a [k][n] stage of block nb at k = 0 (k adds 256 each), and of a [k][m] one
    int boff[4], aoff[NTB];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        boff[i] = BROWS ? (wn * 128 + i * 32 + (lane & 31)) * TR_BK :
                  (8 * fhalf + rr) * TR_BN + (((16 * wn + 4 * i + 2 * g16 + (cc >> 1)) ^ (rr << 2)) << 3) + (cc & 1) * 4;
#pragma unroll
    for (int i = 0; i < NTB; ++i) {
        if constexpr (WG)
            aoff[i] = (8 * fhalf + rr) * BM + (((4 * NTB * wm + 4 * i + 2 * g16 + (cc >> 1)) ^ (rr << 2)) << 3) +
                      (cc & 1) * 4;
        else
            aoff[i] = (wm * (BM / 2) + i * 32 + (lane & 31)) * TR_BK;
    }
    int asw[NTB], bsw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = wn * 128 + i * 32 + (lane & 31);
        bsw[i] = TR_BK == 32 ? (r >> 1) & 3 : pf_swz(r);
    }
#pragma unroll
    for (int i = 0; i < NTB; ++i) {
        const int r = wm * (BM / 2) + i * 32 + (lane & 31);
        asw[i] = TR_BK == 32 ? (r >> 1) & 3 : pf_swz(r);
    }
    struct Frags {
        bf16x8 n[4], m[NTB];
    };
    auto read = [&](const bf16* cA, const bf16* cB, int q, Frags& f) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BROWS)
                f.n[i] = *reinterpret_cast<const bf16x8*>(cB + boff[i] + ((2 * q + fhalf) ^ bsw[i]) * 8);
            else
                f.n[i] = read_tr(cB + boff[i] + 16 * q * TR_BN, cB + boff[i] + (16 * q + 4) * TR_BN);
        }
#pragma unroll
        for (int i = 0; i < NTB; ++i) {
            if constexpr (WG)
                f.m[i] = read_tr(cA + aoff[i] + 16 * q * BM, cA + aoff[i] + (16 * q + 4) * BM);
            else
                f.m[i] = *reinterpret_cast<const bf16x8*>(cA + aoff[i] + ((2 * q + fhalf) ^ asw[i]) * 8);
        }
    };
    constexpr int NM = 4 * NTB;                       // MFMAs of a quarter
    constexpr int NR = (BROWS ? 4 : 8) + (WG ? 2 * NTB : NTB);  // LDS reads of a quarter
    f32x16 acc[4][NTB];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < NTB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.0f;
    auto mma = [&](const Frags& f) __attribute__((always_inline)) {
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < NTB; ++b) acc[a][b] = mfma32(f.n[a], f.m[b], acc[a][b]);
    };
    // One quarter's schedule: reads and NV loads spread over the MFMAs.
    auto weave = [&](auto nv_c) __attribute__((always_inline)) {
        constexpr int NV = decltype(nv_c)::value;
#pragma unroll
        for (int i = 0; i < NM; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            const int nr = ((i + 1) * NR) / NM - (i * NR) / NM, nl = ((i + 1) * NV) / NM - (i * NV) / NM;
#pragma unroll
            for (int l = 0; l < (NR + NM - 1) / NM; ++l)
                if (l < nr) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
#pragma unroll
            for (int l = 0; l < (NV + NM - 1) / NM; ++l)
                if (l < nl) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
    };

    // Stage kt: its four quarters, each overlapping the LDS reads of the next.
    // After the third: this wave's reads of the stage are done and its loads of
    // stage kt + 1 have landed; the barrier then frees the stage's units.
    Frags fa, fb;
    // Five-unit ring: the early operand of stage kt is in unit 2 kt % 5, the late
    // one in the next; early(kt + 2) goes into unit p during the first three
    // quarters, late(kt + 2) into early(kt)'s unit after the barrier.  The early
    // operand is the weights, which stream from HBM (TR_DW: the m side).
    constexpr bool SW = !WG;
    auto step5 = [&](int kt, bf16* c1, bf16* c2, const bf16* n1, const bf16* n2, bf16* p) __attribute__((always_inline)) {
        const bf16 *cA = SW ? c2 : c1, *cB = SW ? c1 : c2, *nA = SW ? n2 : n1, *nB = SW ? n1 : n2;
        const auto ra = rs_a(ks + kt + 2);
        const RsB rb = rs_bs(ks + kt + 2);
        auto early = [&](int j) __attribute__((always_inline)) {
            if constexpr (SW) ld_b(rb.r, ks + kt + 2, j, p);
            else ld_a(ra, ks + kt + 2, j, p);
        };
        static_assert(!RING5 || (NJA == 8 && NJB == 8), "loads of a half");
        read(cA, cB, 1, fb);
#pragma unroll
        for (int j = 0; j < 3; ++j) early(j);
        mma(fa);
        weave(std::integral_constant<int, 3>{});
        __builtin_amdgcn_sched_barrier(0);
        read(cA, cB, 2, fa);
#pragma unroll
        for (int j = 3; j < 6; ++j) early(j);
        mma(fb);
        weave(std::integral_constant<int, 3>{});
        __builtin_amdgcn_sched_barrier(0);
        read(cA, cB, 3, fb);
#pragma unroll
        for (int j = 6; j < 8; ++j) early(j);
        mma(fa);
        weave(std::integral_constant<int, 2>{});
        __builtin_amdgcn_sched_barrier(0);
        PF_WAIT_LGKM0();
        PF_WAIT_VM(8);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (SW) ld_a(ra, ks + kt + 2, j, c1);
            else ld_b(rb.r, ks + kt + 2, j, c1);
        }
        read(nA, nB, 0, fa);
        mma(fb);
        weave(std::integral_constant<int, 8>{});
        __builtin_amdgcn_sched_barrier(0);
    };
    // Stage kt + 2 into slot (kt + 2) % 3, half of its loads in each of the
    // stage's two 16-wide parts (L; the first stage's step finds them on the way).
    auto step3 = [&](auto l_c, int kt, bf16* cA, bf16* cB, const bf16* nA, const bf16* nB, bf16* pA, bf16* pB) __attribute__((always_inline)) {
        constexpr bool L = decltype(l_c)::value;
        constexpr int V = NLD / 2;
        const auto ra = rs_a(ks + kt + 2);
        const RsB rb = rs_bs(ks + kt + 2);
        auto lds = [&](int i0) __attribute__((always_inline)) {
#pragma unroll
            for (int i = i0; i < i0 + V; ++i) {
                if (i < NJA) ld_a(ra, ks + kt + 2, i, pA);
                else ld_b(rb.r, ks + kt + 2, i - NJA, pB);
            }
        };
        read(cA, cB, 1, fb);
        if constexpr (L) lds(0);
        mma(fa);
        weave(std::integral_constant<int, L ? V : 0>{});
        __builtin_amdgcn_sched_barrier(0);
        PF_WAIT_LGKM0();
        PF_WAIT_VM(L ? V : NLD);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (L) lds(V);
        read(nA, nB, 0, fa);
        mma(fb);
        weave(std::integral_constant<int, L ? V : 0>{});
        __builtin_amdgcn_sched_barrier(0);
    };
    auto first = [&](int kt, bf16* dA, bf16* dB) __attribute__((always_inline)) {
        const auto ra = rs_a(ks + kt);
        const RsB rb = rs_bs(ks + kt);
#pragma unroll
        for (int j = 0; j < NJA; ++j) ld_a(ra, ks + kt, j, dA);
#pragma unroll
        for (int j = 0; j < NJB; ++j) ld_b(rb.r, ks + kt, j, dB);
    };
    if (nk > 0) {
        if constexpr (RING5) {
            bf16 *const u0 = sA0, *const u1 = sB0, *const u2 = sA1, *const u3 = sB1, *const u4 = sU4;
            first(0, SW ? u1 : u0, SW ? u0 : u1);
            first(1, SW ? u3 : u2, SW ? u2 : u3);
            PF_WAIT_VM(NLD);
            __builtin_amdgcn_s_barrier();
            read(SW ? u1 : u0, SW ? u0 : u1, 0, fa);
            const int main = nk - nk % 5;
            for (int k = 0; k < main; k += 5) {
                step5(k, u0, u1, u2, u3, u4);
                step5(k + 1, u2, u3, u4, u0, u1);
                step5(k + 2, u4, u0, u1, u2, u3);
                step5(k + 3, u1, u2, u3, u4, u0);
                step5(k + 4, u3, u4, u0, u1, u2);
            }
            const int rem = nk - main;
            if (rem > 0) step5(main, u0, u1, u2, u3, u4);
            if (rem > 1) step5(main + 1, u2, u3, u4, u0, u1);
            if (rem > 2) step5(main + 2, u4, u0, u1, u2, u3);
            if (rem > 3) step5(main + 3, u1, u2, u3, u4, u0);
        } else {
            constexpr std::true_type L{};
            first(0, sA0, sB0);
            first(1, sA1, sB1);
            first(2, sA2, sB2);
            PF_WAIT_VM(2 * NLD);
            __builtin_amdgcn_s_barrier();
            read(sA0, sB0, 0, fa);
            step3(std::false_type{}, 0, sA0, sB0, sA1, sB1, nullptr, nullptr);
            const int rem = (nk - 1) % 3, main = nk - rem;
            for (int k = 1; k < main; k += 3) {
                step3(L, k, sA1, sB1, sA2, sB2, sA0, sB0);
                step3(L, k + 1, sA2, sB2, sA0, sB0, sA1, sB1);
                step3(L, k + 2, sA0, sB0, sA1, sB1, sA2, sB2);
            }
            if (rem > 0) step3(L, main, sA1, sB1, sA2, sB2, sA0, sB0);
            if (rem > 1) step3(L, main + 1, sA2, sB2, sA0, sB0, sA1, sB1);
        }
    }
    PF_WAIT_VM(0);
    PF_WAIT_LGKM0();
    __builtin_amdgcn_s_barrier();  // no wave reads the ring any more
    __builtin_amdgcn_sched_barrier(0);

    // ---- epilogue --------------------------------------------------------------------
    // acc[nb][mb][i]: column wn * 128 + 32 nb + 8 (i / 4) + 4 (lane / 32) + i % 4,
    // row wm * BM / 2 + 32 mb + lane % 32.  Each wave passes its block through an
    // LDS unit of its own (chunks swizzled by row) and writes 16 bytes per lane.
    bf16* const st = RING5 ? (wave == 0 ? sB0 : wave == 1 ? sB1 : wave == 2 ? sA0 : sA1)
                           : (wave == 0 ? sB0 : wave == 1 ? sB1 : wave == 2 ? sB2 : sA0);
    const int mrow = wm * (BM / 2), ncol = n0 + wn * 128;
    const int el = pf_lane_fresh();
    if constexpr (PART) {
        // fp32 sums, 32 rows x 64 columns (8 KB) at a time
        float* const sf = reinterpret_cast<float*>(st);
        // of the range: result e * sels + (which of them), or all rows
        float* const dst = WG ? g.part + (((size_t)range * g.E + e) * 3 + sel) * M * N
                              : g.part + (size_t)range * g.n_rows * N;
        const int r0 = WG ? m0 : row0, r_end = WG ? M : row_end;
        const int lrow = el >> 4, lch = el & 15;
#pragma unroll
        for (int p = 0; p < 2 * NTB; ++p) {
            const int mb = p >> 1, half = p & 1;
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int ch = nb * 8 + 2 * q + (el >> 5), rl = el & 31;
                    const f32x16& a = acc[2 * half + nb][mb];
                    *reinterpret_cast<f32x4*>(sf + rl * 64 + ((ch ^ (rl & 15)) << 2)) =
                        f32x4{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
                }
            const int c = ncol + half * 64 + lch * 4;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int rl = i * 4 + lrow, r = r0 + mrow + mb * 32 + rl;
                const f32x4 v = *reinterpret_cast<const f32x4*>(sf + rl * 64 + ((lch ^ (rl & 15)) << 2));
                if (r < r_end && c < N) *reinterpret_cast<f32x4*>(dst + (size_t)r * N + c) = v;
            }
        }
    } else if constexpr (MODE == TR_DACT) {
        // fp32 sums, 32 rows x 64 columns (8 KB) at a time; then gate and up by whole lines
        float* const sf = reinterpret_cast<float*>(st);
        const int lrow = el >> 3, lch = el & 7;  // eight chunks of eight columns per row
        bf16x8 gv[2][4], uv[2][4];  // a pass's gate and up, loaded one pass ahead
        auto fetch = [&](int p) __attribute__((always_inline)) {
            const int c = min(ncol + (p & 1) * 64 + lch * 8, N - 8);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = min(row0 + mrow + (p >> 1) * 32 + i * 8 + lrow, row_end - 1);
                gv[p & 1][i] = *reinterpret_cast<const bf16x8*>(g.gate + (size_t)r * N + c);
                uv[p & 1][i] = *reinterpret_cast<const bf16x8*>(g.up + (size_t)r * N + c);
            }
        };
        fetch(0);
#pragma unroll
        for (int p = 0; p < 2 * NTB; ++p) {
            const int mb = p >> 1, half = p & 1;
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int ch = nb * 8 + 2 * q + (el >> 5), rl = el & 31;
                    const f32x16& a = acc[2 * half + nb][mb];
                    *reinterpret_cast<f32x4*>(sf + rl * 64 + ((ch ^ (rl & 15)) << 2)) =
                        f32x4{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
                }
            if (p + 1 < 2 * NTB) fetch(p + 1);
            const int c = ncol + half * 64 + lch * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int rl = i * 8 + lrow, r = row0 + mrow + mb * 32 + rl;
                const f32x4 d0 = *reinterpret_cast<const f32x4*>(sf + rl * 64 + (((2 * lch) ^ (rl & 15)) << 2));
                const f32x4 d1 = *reinterpret_cast<const f32x4*>(sf + rl * 64 + (((2 * lch + 1) ^ (rl & 15)) << 2));
                bf16x8 o0, o1, o2;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const GatedGrad v =
                        gated_grad((float)gv[p & 1][i][j], (float)uv[p & 1][i][j], j < 4 ? d0[j & 3] : d1[j & 3]);
                    o0[j] = (bf16)v.dg;
                    o1[j] = (bf16)v.du;
                    o2[j] = (bf16)v.act;
                }
                if (r < row_end && c < N) {
                    const size_t at = (size_t)r * N + c;
                    *reinterpret_cast<bf16x8*>(g.out0 + at) = o0;
                    *reinterpret_cast<bf16x8*>(g.out1 + at) = o1;
                    *reinterpret_cast<bf16x8*>(g.out2 + at) = o2;
                }
            }
        }
    } else if constexpr (MODE == TR_GATE) {
        // blocks 0 and 2 hold gate sums, 1 and 3 the up sums of the same 32
        // features: act, gate and up in turn, the wave's rows x 64 features each
        const int lrow = el >> 3, lch = el & 7;
        const int c = n0 + wn * 64 + lch * 8;
#pragma unroll
        for (int which = 0; which < 3; ++which) {
            bf16* const dst = which == 0 ? g.out0 : which == 1 ? g.out1 : g.out2;
#pragma unroll
            for (int mb = 0; mb < NTB; ++mb)
#pragma unroll
                for (int pr = 0; pr < 2; ++pr)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int rl = mb * 32 + (el & 31), cl = pr * 32 + 8 * q + 4 * (el >> 5);
                        const f32x16 &ga = acc[2 * pr][mb], &ua = acc[2 * pr + 1][mb];
                        bf16x4 o;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float gv = ga[4 * q + j], uv = ua[4 * q + j];
                            o[j] = (bf16)(which == 0 ? silu(gv) * uv : which == 1 ? gv : uv);
                        }
                        *reinterpret_cast<bf16x4*>(st + rl * 64 + (((cl >> 3) ^ (rl & 7)) << 3) + (cl & 7)) = o;
                    }
#pragma unroll
            for (int i = 0; i < NTB * 4; ++i) {
                const int rl = i * 8 + lrow, r = row0 + mrow + rl;
                const bf16x8 v = *reinterpret_cast<const bf16x8*>(st + rl * 64 + ((lch ^ (rl & 7)) << 3));
                if (r < row_end && c < N) *reinterpret_cast<bf16x8*>(dst + (size_t)r * N + c) = v;
            }
        }
    } else {
        // in passes of the rows that a unit holds
        constexpr int PB = RING5 ? NTB : 1;  // 32-row blocks per pass
        const int lrow = el >> 4, lch = el & 15;  // 16 chunks of eight columns per row
        const int r_end = WG ? M : row_end, r0 = (WG ? m0 : row0) + mrow;
        const int c = ncol + lch * 8;
#pragma unroll
        for (int p = 0; p < NTB; p += PB) {
#pragma unroll
            for (int mb = p; mb < p + PB; ++mb) {
                const int rl = (mb - p) * 32 + (el & 31);
#pragma unroll
                for (int nb = 0; nb < 4; ++nb)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int cl = nb * 32 + 8 * q + 4 * (el >> 5);
                        *reinterpret_cast<bf16x4*>(st + rl * 128 + (((cl >> 3) ^ (rl & 7)) << 3) + (cl & 7)) =
                            bf16x4{(bf16)acc[nb][mb][4 * q], (bf16)acc[nb][mb][4 * q + 1], (bf16)acc[nb][mb][4 * q + 2],
                                   (bf16)acc[nb][mb][4 * q + 3]};
                    }
            }
#pragma unroll
            for (int i = 0; i < PB * 8; ++i) {
                const int rl = i * 4 + lrow, r = r0 + p * 32 + rl;
                const bf16x8 v = *reinterpret_cast<const bf16x8*>(st + rl * 128 + ((lch ^ (rl & 7)) << 3));
                if (r < r_end && c < N) {
                    bf16x8* const q = reinterpret_cast<bf16x8*>(out + (size_t)r * N + c);
                    // a gradient is not read again here: past the caches, which keep the
                    // operands (32 experts of 128 rows: the backward pass 1.51 -> 1.42 ms)
                    if constexpr (WG) __builtin_nontemporal_store(v, q);
                    else *q = v;
                }
            }
        }
    }
}

template <int MODE, bool KT>
hipError_t launch_tiles(const TrainArgs& g, int bm, unsigned grid, hipStream_t s) {
    if (bm == 256) ffn_train_kernel<MODE, 256, KT><<<grid, 256, 0, s>>>(g);
    else ffn_train_kernel<MODE, 128, KT><<<grid, 256, 0, s>>>(g);
    return hipGetLastError();
}

// Adds the ranges of rows in order; result blockIdx.y of 3 E.
__global__ __launch_bounds__(256) void dw_reduce_kernel(size_t n, int parts, const float* __restrict__ part,
                                                       bf16* __restrict__ out0, bf16* __restrict__ out1,
                                                       bf16* __restrict__ out2) {
    const int res = blockIdx.y, sel = res % 3;
    const float* src = part + (size_t)res * n;
    bf16* dst = (sel == 0 ? out0 : sel == 1 ? out1 : out2) + (size_t)(res / 3) * n;
    const size_t step = (size_t)gridDim.y * n;
    for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (size_t)gridDim.x * 1024) {
        f32x4 v = *reinterpret_cast<const f32x4*>(src + i);
        for (int p = 1; p < parts; ++p) v += *reinterpret_cast<const f32x4*>(src + p * step + i);
        *reinterpret_cast<bf16x4*>(dst + i) = bf16x4{(bf16)v[0], (bf16)v[1], (bf16)v[2], (bf16)v[3]};
    }
}

// TR_DX, TR_DOWN: adds the ranges of stages of the rows before *live (the groups' end).
__global__ __launch_bounds__(256) void rows_reduce_kernel(int n_rows, int N, int parts, const float* __restrict__ part,
                                                         const int32_t* __restrict__ live, bf16* __restrict__ out) {
    const size_t n = (size_t)min(n_rows, *live) * N, step = (size_t)n_rows * N;
    for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (size_t)gridDim.x * 1024) {
        f32x4 v = *reinterpret_cast<const f32x4*>(part + i);
        for (int p = 1; p < parts; ++p) v += *reinterpret_cast<const f32x4*>(part + p * step + i);
        *reinterpret_cast<bf16x4*>(out + i) = bf16x4{(bf16)v[0], (bf16)v[1], (bf16)v[2], (bf16)v[3]};
    }
}

// Ranges of the stages of a product of n rows and N columns over K: with few
// tiles, enough for two workgroups per compute unit, eight stages or more each
// (two experts of 24 rows, d 88, F 2944: the backward pass 94 -> 45 us).
int row_ranges(int n, int E, int N, int K, int bm) {
    if (bm != 128) return 1;
    const long tiles = (long)row_plan_tiles(n, E, 128) * ((N + TR_BN - 1) / TR_BN);
    return (int)std::max(1L, std::min(std::min(512 / tiles, (long)K / 256), 16L));
}
size_t row_part_bytes(int n, int E, int N, int K) {
    const int parts = row_ranges(n, E, N, K, 128);
    return parts > 1 ? (size_t)parts * n * N * sizeof(float) : 0;
}

// Slots of one expert's results per XCD (TR_DW).
long dw_slots(int d, int F, int bm) {
    const auto per = [&](int m, int n) {
        return ((long)((m + bm - 1) / bm) * ((n + TR_BN - 1) / TR_BN) + PF_XCD - 1) / PF_XCD;
    };
    return per(d, F) + 2 * per(F, d);
}

// Ranges that the rows of TR_DW are cut into: with few result tiles and long
// groups, enough for two workgroups per compute unit, 512 rows or more each
// (one expert of 6244 rows, d 520, F 152: the backward pass 242 -> 75 us).
int dw_ranges(int n, int E, int d, int F) {
    const long tiles = ((long)((d + 127) / 128) * ((F + TR_BN - 1) / TR_BN) +
                        2L * ((F + 127) / 128) * ((d + TR_BN - 1) / TR_BN)) * E;
    return (int)std::max(1L, std::min(512 / tiles, (long)n / E / 512));
}
size_t dw_part_bytes(int n, int E, int d, int F) {
    const int parts = dw_ranges(n, E, d, F);
    return parts > 1 ? (size_t)parts * 3 * E * d * F * sizeof(float) : 0;
}

// dW2 = dh^T act, dW1 = dgate^T x and dW3 = dup^T x of every expert, in one launch.
hipError_t launch_dw(int n, int E, int d, int F, const bf16* dh, const bf16* act, const bf16* dgate, const bf16* dup,
                     const bf16* x, bf16* dw2, bf16* dw1, bf16* dw3, const int32_t* offsets, float* part,
                     hipStream_t s) {
    TrainArgs g{};
    g.a0 = dh;
    g.b0 = act;
    g.out0 = dw2;
    g.a1 = dgate;
    g.a2 = dup;
    g.b1 = g.b2 = x;
    g.out1 = dw1;
    g.out2 = dw3;
    g.n_rows = n;
    g.E = E;
    g.M = g.lda = d;
    g.N = g.ldb = F;
    g.offsets = offsets;
    g.parts = dw_ranges(n, E, d, F);
    g.part = part;
    const int bm = g.parts == 1 && n >= TR_DW_LONG * E ? 256 : 128;
    const unsigned grid = (unsigned)(dw_slots(d, F, bm) * E * g.parts * PF_XCD);
    if (g.parts == 1) return launch_tiles<TR_DW, false>(g, bm, grid, s);
    ffn_train_kernel<TR_DW, 128, false, true><<<grid, 256, 0, s>>>(g);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const size_t each = (size_t)d * F;
    dw_reduce_kernel<<<dim3((unsigned)std::min<size_t>((each + 1023) / 1024, 1024), 3 * E), 256, 0, s>>>(
        each, g.parts, part, dw2, dw1, dw3);
    return hipGetLastError();
}

}  // namespace

// Row tiles: 256 from 128 rows per expert on (padded halves cost little where
// the weights are the bound: 32 experts of 128 rows, d 7168, F 2048: da 253 ->
// 203 us, dx 507 -> 467), else 128, and 128 too where 256 would leave compute
// units idle (cols: the narrower product's columns).
static int train_bm(int n, int E, int cols) {
    return n >= 128 * E && (long)row_plan_tiles(n, E, 256) * ((cols + TR_BN - 1) / TR_BN) >= 256 ? 256 : 128;
}
static unsigned train_grid(int n, int E, int bm, int n_nt) {
    return (unsigned)(((long)row_plan_tiles(n, E, bm) * n_nt + PF_XCD - 1) / PF_XCD * PF_XCD);
}

// A product over rows whose sum may be cut into ranges (K: of one product).
template <int MODE>
static hipError_t launch_rows(TrainArgs& g, int bm, int ranges, float* part, hipStream_t s) {
    const unsigned grid = train_grid(g.n_rows, g.E, bm, g.n_nt * ranges);
    if (ranges == 1) {
        if constexpr (MODE == TR_DX)
            if (g.K % 64 == 0) return launch_tiles<MODE, false>(g, bm, grid, s);
        return launch_tiles<MODE, true>(g, bm, grid, s);
    }
    g.parts = ranges;
    g.part = part;
    ffn_train_kernel<MODE, 128, true, true><<<grid, 256, 0, s>>>(g);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const size_t vecs = (size_t)g.n_rows * g.N / 4;
    rows_reduce_kernel<<<(unsigned)std::min<size_t>((vecs + 255) / 256, 2048), 256, 0, s>>>(
        g.n_rows, g.N, ranges, part, g.offsets + g.E, g.out0);
    return hipGetLastError();
}

size_t ffn_train_tiles_ws_bytes(int n, int E, int d, int F) { return row_plan_bytes(n, E) + row_part_bytes(n, E, d, F); }

hipError_t launch_ffn_train_tiles(int n, int E, int d, int F, const bf16* x, const int32_t* offsets, const bf16* w1,
                                  const bf16* w3, const bf16* w2, bf16* gate, bf16* up, bf16* act, bf16* h, void* ws,
                                  hipStream_t s) {
    const int bm = train_bm(n, E, std::min(d, F));
    TrainArgs g{};
    hipError_t err = hipSuccess;
    if (E > GroupTiles::kMax) err = launch_row_plan(n, E, bm, offsets, ws, &g.plan, s);
    if (err != hipSuccess) return err;
    g.n_rows = n;
    g.E = E;
    g.offsets = offsets;
    g.a0 = x;
    g.b0 = w1;
    g.b1 = w3;
    g.out0 = act;
    g.out1 = gate;
    g.out2 = up;
    g.N = F;
    g.K = g.lda = g.ldb = d;
    g.n_nt = (F + 127) / 128;
    if ((err = launch_tiles<TR_GATE, true>(g, bm, train_grid(n, E, bm, g.n_nt), s)) != hipSuccess) return err;
    g.a0 = act;
    g.b0 = w2;
    g.out0 = h;
    g.N = d;
    g.K = g.lda = g.ldb = F;
    g.n_nt = (d + TR_BN - 1) / TR_BN;
    return launch_rows<TR_DOWN>(g, bm, row_ranges(n, E, d, F, bm),
                                reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + row_plan_bytes(n, E)), s);
}

// The row plan, then the ranges' sums of one product after the other.
size_t ffn_grad_ws_bytes(int n, int E, int d, int F) {
    return row_plan_bytes(n, E) + std::max(dw_part_bytes(n, E, d, F), row_part_bytes(n, E, d, 2 * F));
}

hipError_t launch_ffn_grad(int n, int E, int d, int F, const bf16* x, const int32_t* offsets, const bf16* w1,
                           const bf16* w3, const bf16* w2, const bf16* gate, const bf16* up, const bf16* dh, bf16* dx,
                           bf16* dw1, bf16* dw3, bf16* dw2, bf16* dgate, bf16* dup, bf16* act, void* ws,
                           hipStream_t s) {
    const int bm = train_bm(n, E, std::min(d, F));
    RowPlan plan;
    hipError_t err = hipSuccess;
    if (E > GroupTiles::kMax) err = launch_row_plan(n, E, bm, offsets, ws, &plan, s);
    if (err != hipSuccess) return err;
    float* part = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + row_plan_bytes(n, E));
    auto grid = [&](int n_nt) { return train_grid(n, E, bm, n_nt); };
    TrainArgs g{};
    g.a0 = dh;
    g.b0 = w2;
    g.out0 = dgate;
    g.out1 = dup;
    g.out2 = act;
    g.gate = gate;
    g.up = up;
    g.n_rows = n;
    g.E = E;
    g.N = g.ldb = F;
    g.K = g.lda = d;
    g.n_nt = (F + TR_BN - 1) / TR_BN;
    g.plan = plan;
    g.offsets = offsets;
    err = d % 64 == 0 ? launch_tiles<TR_DACT, false>(g, bm, grid(g.n_nt), s)
                         : launch_tiles<TR_DACT, true>(g, bm, grid(g.n_nt), s);
    if (err != hipSuccess) return err;
    if (dw2 != nullptr) {
        err = launch_dw(n, E, d, F, dh, act, dgate, dup, x, dw2, dw1, dw3, offsets, part, s);
        if (err != hipSuccess) return err;
    }
    if (dx != nullptr) {
        g.a0 = dgate;
        g.a1 = dup;
        g.b0 = w1;
        g.b1 = w3;
        g.out0 = dx;
        g.N = g.ldb = d;
        g.K = g.lda = F;
        g.n_nt = (d + TR_BN - 1) / TR_BN;
        err = launch_rows<TR_DX>(g, bm, row_ranges(n, E, d, 2 * F, bm), part, s);
    }
    return err;
}

}  // namespace moe
