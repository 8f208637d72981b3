// ssd_linear_plan.h -- which tile of ssd_linear.h a matrix product takes, and how its operands' rows come to it (host code
// alone, of sizes and types).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

namespace ssd {

// Operands of the product: rows with the contraction's values one behind the other.
// LT_E4M3_F32: e4m3 for outputs in fp32 (a kernel's type; everywhere else LT_E4M3).
enum : int { LT_F32 = 0, LT_F16 = 1, LT_BF16 = 2, LT_I8 = 3, LT_E4M3 = 4, LT_E4M3_F32 = 5 };
struct LinearPlan {
    int tile;    // index of the tile shape
    int splits;  // of the contraction
    float us;    // by the model that chose them
    bool narrow; // loads of 4 bytes a lane: rows of a multiple of 4 bytes
};
struct LinearSize {
    int64_t M, N, kbytes;
    LinearPlan plan;
};

// The tile and the splits of the contraction by a model of the time, fitted to sweeps over 1 to 8192 rows at 2560 x
// 10576, 5120 x 2560, 1024 x 4096, 4096 x 1024 and 8192 x 8192 (bf16: of 19 such products it takes the fastest pair of the
// sweep or one within 11 %, but for 64 x 2560 x 10576, 24 us against 19; the other types have the same constants: of ten products
// of 1 to 8192 rows fp16, int8 and e4m3 take the fastest or one within 9 %, but for these 64 rows in fp16, fp32 one within
// 15 %, but for 128 x 2560 x 10576 and 512 x 5120 x 2560, 93 and 155 us against 74 and 123):
//   2.5 us + rounds (steps c + e),  and 4 us + 8 bytes a partial sum at 4 TB/s where the contraction is split,
// c being the time of a step with 1, 2, .. workgroups a CU and e that of a tile's start and epilogue.  8192 x 5120 x 2560
// takes 206 us in tiles of 256 x 160 (two full rounds of 256 CUs), 271 us in 256 x 256 and 248 us in 128 x 128; 16 x
// 5120 x 2560 10.9 us in 16 x 64 split by 4, 13.5 us unsplit.  fp32 is bound by its matrix instructions, 16 times slower: c
// goes by the area, down to what a step's latency takes.
// Rows that are no multiple of 16 bytes are copied to ones that are (3 us and their bytes twice at 4 TB/s), or, of a multiple
// of 4 bytes and in the three smaller tiles, loaded by 4 bytes a lane, whose steps take 1.35 times as long: one row of 2562
// x 10576 bf16 14.2 us against 35.6 copied, 16 rows 18.7 and 36.4, 128 rows 37 and 47; but fp32 1500 x 1110 x 2000 88 and 77.
struct TileModel {
    uint32_t bm, bn;
    int most;  // workgroups a CU
    float c[2], e;
};
constexpr TileModel kTiles[] = {
    {128, 128, 2, {0.75f, 0.90f}, 4.f}, {256, 256, 1, {1.67f, 0.f}, 6.f},    {128, 192, 2, {0.85f, 1.28f}, 5.f},
    {256, 160, 1, {1.15f, 0.f}, 5.f},   {256, 128, 1, {0.88f, 0.f}, 5.f},    {64, 128, 2, {0.45f, 0.60f}, 2.5f},
    {32, 64, 2, {0.17f, 0.30f}, 2.f},   {16, 64, 2, {0.165f, 0.28f}, 2.f},   {128, 128, 1, {0.50f, 0.f}, 4.f},
};
constexpr int kTileCount = sizeof(kTiles) / sizeof(kTiles[0]);
constexpr uint32_t kCUs = 256;

// The time of `groups` workgroups of so many steps, `longest` of one of them.
inline float tiles_us(const TileModel& m, int type, int64_t groups, float steps, float longest = 0.f) {
    const int o = m.most > 1 && groups > kCUs ? 2 : 1;
    const float f32 = 1.95f / 16384.f * (float)(o * m.bm * m.bn), c = type != LT_F32 ? m.c[o - 1] : f32 > 0.2f ? f32 : 0.2f;
    const float all = (float)((groups + kCUs * o - 1) / (kCUs * o)) * (steps * c + m.e), one = longest * c + m.e;
    return all > one ? all : one;
}
inline int64_t tiles_of(const TileModel& m, int64_t M, int64_t N) {
    return (int64_t)(((uint32_t)M + m.bm - 1) / m.bm) * (((uint32_t)N + m.bn - 1) / m.bn);
}
constexpr int64_t kMostGroups = ((int64_t)1 << 32) / 512;  // (lanes of a launch; 256 x 256 always fits)

// copied: the bytes of rows that 16-byte loads do not take as they are, to be copied first (plan not narrow) or loaded by 4
// bytes; may_narrow: whether these can be
inline LinearPlan linear_plan(int64_t M, int64_t N, int64_t kbytes, int type, int64_t copied = 0, bool may_narrow = false) {
    const int64_t steps = (kbytes + 127) / 128;
    LinearPlan best{0, 1, 3.4e38f, false};
    const auto splitting = [&](int splits) { return splits > 1 ? 4.f + (float)splits * (float)M * (float)N * 2e-6f : 0.f; };
    int64_t tiles[kTileCount];
    for (int t = 0; t < kTileCount; ++t) tiles[t] = tiles_of(kTiles[t], M, N);
    for (int splits : {1, 2, 3, 4, 6, 8, 12, 16}) {
        const uint32_t per = ((uint32_t)steps + splits - 1) / splits;
        if (splits > 1 && (per < 4 || ((uint32_t)steps + per - 1) / per != (uint32_t)splits)) break;  // (none without a step)
        const float rest = 2.5f + splitting(splits);
        if (rest >= best.us) break;
        for (int t = 0; t < kTileCount; ++t) {
            if (tiles[t] * splits >= kMostGroups) continue;
            const float us = rest + tiles_us(kTiles[t], type, tiles[t] * splits, (float)per);
            if (us < best.us) best = LinearPlan{t, splits, us, false};
        }
    }
    if (!copied) return best;
    best.us += 3.f + (float)copied * 0.5e-6f;
    if (!may_narrow) return best;
    // (the same splits, so that the same values give the same sums to the bit in rows of any alignment)
    const int splits = best.splits;
    const int64_t per = (steps + splits - 1) / splits;
    for (int t = 5; t <= 7; ++t) {
        const int64_t groups = tiles[t] * splits;
        if (groups >= kMostGroups) continue;
        const float us = 2.5f + tiles_us(kTiles[t], type, groups, (float)per * 1.35f) + splitting(splits);
        if (us < best.us) best = LinearPlan{t, splits, us, true};
    }
    return best;
}

// Two products in one launch, where their tiles fill the chip better than each product's alone (4096 x 4096 x 1024 twice,
// f16: 65 us in 256 tiles of 256 x 128, 2 x 39 us in 128 x 128): the tile, by the same model, with the average of the
// workgroups' steps, and no less than the longest takes.  (Products of unlike contractions go one by one: 512 x 2560 x 10576,
// f16, takes 90 us so, 260 in one launch of 256 x 256.)  Splits 0: one by one is as fast.
inline LinearPlan linear_plan_two(const LinearSize& a, const LinearSize& b, int type) {
    LinearPlan best{0, 0, a.plan.us + b.plan.us, false};
    const float sa = (float)((a.kbytes + 127) / 128), sb = (float)((b.kbytes + 127) / 128);
    for (int t = 0; t < kTileCount; ++t) {
        const int64_t ta = tiles_of(kTiles[t], a.M, a.N), tb = tiles_of(kTiles[t], b.M, b.N);
        if (ta + tb >= kMostGroups) continue;
        const float mean = ((float)ta * sa + (float)tb * sb) / (float)(ta + tb);
        const float us = 2.5f + tiles_us(kTiles[t], type, ta + tb, mean, sa > sb ? sa : sb);
        if (us < best.us) best = LinearPlan{t, 1, us, false};
    }
    return best;
}

// ---- operands ------------------------------------------------------------------------------------
constexpr int64_t kMaxRowBytes = (int64_t)1 << 22;  // of an operand: 256 rows of a tile have 31-bit offsets

// K values as rows of 16-byte pieces.
inline int64_t padded(int64_t k, size_t es) {
    const int64_t per = 16 / (int64_t)es;
    return (k + per - 1) / per * per;
}
inline bool rows_fit(int64_t stride, size_t es, size_t piece) {
    return stride * es % piece == 0 && stride * (int64_t)es < kMaxRowBytes;
}

// A product: which operands are copied, to rows of kp values.
struct LinearForm {
    LinearPlan plan;
    bool pack_x, pack_w, may_pack_x;
    int64_t kp;
};
// x_stride: elements between rows of x, 0: contiguous ones
inline LinearForm linear_form(int64_t M, int64_t K, int64_t N, int64_t x_stride, int type, size_t es) {
    LinearForm l{};
    const int64_t xs = x_stride ? x_stride : K;
    l.kp = padded(K, es);
    l.pack_w = l.kp != K;
    l.pack_x = l.kp != K || !rows_fit(xs, es, 16);
    l.may_pack_x = l.pack_x || x_stride;  // a view's rows, also of one row, may start anywhere
    const int64_t copied = ((l.pack_x ? M : 0) + (l.pack_w ? N : 0)) * K * (int64_t)es;
    l.plan = linear_plan(M, N, l.kp * es, type, copied, rows_fit(K, es, 4) && rows_fit(xs, es, 4));
    if (l.plan.narrow) l.pack_w = l.pack_x = false;
    return l;
}

// Its gradients' two products, over rows of np and mp values.
struct LinearBackForm {
    LinearPlan dx_plan, dw_plan, both_plan;  // (both: splits 0 where they are launched one by one)
    int64_t mp, np;
};
inline LinearBackForm linear_back_form(int64_t M, int64_t K, int64_t N, int type, size_t es) {
    LinearBackForm l{};
    l.mp = padded(M, es);
    l.np = padded(N, es);
    const int64_t eb = es;
    l.dx_plan = linear_plan(M, K, l.np * eb, type);
    l.dw_plan = linear_plan(N, K, l.mp * eb, type);
    l.both_plan = linear_plan_two({M, K, l.np * eb, l.dx_plan}, {N, K, l.mp * eb, l.dw_plan}, type);
    return l;
}

}  // namespace ssd
