// rope.cuh -- the angles of rotary positions.
//
// Pair i of a head turns by pos * f_i.  f_i / (2 pi), turns per position, is kept as a
// 64-bit fraction of a turn, so the product with a position, wrapping as integers do, is the
// angle within its turn to pos * 2^-65 turns, however far the position: in f32 the angle of
// position 131072 would be off by 0.004 radians.
//
// Cosine and sine are the f32 numbers next to the true ones (off by 2^-33 before that
// rounding, so another number comes out for one angle in some hundred), and the products and
// sums of a rotation are rounded one by one.  What is held in few bits after a rotation, the
// codes of the 4-bit cache, then depends on the inputs alone and not on how a kernel lays its
// work out.
#pragma once

#include <cstdint>

namespace mmq {

struct RopeView {
    const unsigned long long* turns;   // [rot / 2], fraction of a turn per position, times 2^64
    int rot;                           // values of a head that turn, even
    bool interleaved;                  // pairs (2 i, 2 i + 1), else (i, i + rot / 2)
    float magnitude;                   // of cosine and sine
};

// (cos, sin) of phase / 2^64 turns.  The angle is brought within an eighth of a turn of a
// multiple of a quarter; there, with x = hi + lo its radians and z = x^2,
//   sin x = x + x z (-1/6 + z (1/120 - ...)),  cos x = 1 - z/2 + z^2 (1/24 - z (1/720 - ...)),
// the Taylor series up to x^11 and x^12 (below 2^-36 of what is left out), whose leading
// terms are kept as sums of two f32 numbers (T. J. Dekker, Numer. Math. 18, 1971).
__device__ __forceinline__ float2 rope_cos_sin(unsigned long long phase)
{
    const unsigned long long turned = phase + (1ull << 61);
    const unsigned int quarter = static_cast<unsigned int>(turned >> 62);
    const long long rem = static_cast<long long>(turned & ((1ull << 62) - 1)) - (1ll << 61);   // 2^61: an eighth
    // rem = (fh + fl) 2^31, fh of 24 bits
    const int h = static_cast<int>(rem >> 31);
    const float fh = __int2float_rn(h);
    const float fl = __fmaf_rn(__int2float_rn(static_cast<int>(rem & 0x7fffffff)), 4.656612873077393e-10f,
                               __int2float_rn(h - __float2int_rn(fh)));
    // times pi 2^-32, in two parts
    constexpr float PI_HI = 3.1415927410125732f * 2.3283064365386963e-10f;
    constexpr float PI_LO = -8.742277657347586e-8f * 2.3283064365386963e-10f;
    const float p = __fmul_rn(fh, PI_HI);
    const float q = __fadd_rn(__fmaf_rn(fh, PI_HI, -p), __fmaf_rn(fh, PI_LO, __fmul_rn(fl, PI_HI)));
    const float xh = __fadd_rn(p, q), xl = __fadd_rn(__fsub_rn(p, xh), q);
    const float zh = __fmul_rn(xh, xh);
    const float zl = __fmaf_rn(__fadd_rn(xh, xh), xl, __fmaf_rn(xh, xh, -zh));

    constexpr float S_HI = -0.16666667163372040f, S_LO = 4.967053879312289e-9f;   // -1/6
    float t = __fmaf_rn(zh, -2.5052108385441720e-8f, 2.7557319223985893e-6f);
    t = __fmaf_rn(zh, t, -1.9841269841269841e-4f);
    t = __fmaf_rn(zh, t, 8.3333333333333333e-3f);
    t = __fmul_rn(zh, t);
    const float sh = __fadd_rn(S_HI, t), sl = __fadd_rn(__fadd_rn(__fsub_rn(S_HI, sh), t), S_LO);
    const float wh = __fmul_rn(zh, sh);
    const float wl = __fadd_rn(__fmaf_rn(zh, sh, -wh), __fmaf_rn(zh, sl, __fmul_rn(zl, sh)));
    const float uh = __fmul_rn(xh, wh);
    const float ul = __fadd_rn(__fmaf_rn(xh, wh, -uh), __fmaf_rn(xh, wl, __fmul_rn(xl, wh)));
    float r = __fadd_rn(xh, uh);
    const float sine = __fadd_rn(r, __fadd_rn(__fadd_rn(__fsub_rn(xh, r), uh), __fadd_rn(xl, ul)));

    constexpr float C_HI = 4.1666667908430099e-2f, C_LO = -1.2417634698280722e-9f;   // 1/24
    float v = __fmaf_rn(zh, 2.0876756987868099e-9f, -2.7557319223985891e-7f);
    v = __fmaf_rn(zh, v, 2.4801587301587302e-5f);
    v = __fmaf_rn(zh, v, -1.3888888888888889e-3f);
    v = __fmul_rn(zh, v);
    const float ch = __fadd_rn(C_HI, v), cl = __fadd_rn(__fadd_rn(__fsub_rn(C_HI, ch), v), C_LO);
    const float gh = __fmul_rn(zh, zh);
    const float gl = __fmaf_rn(__fadd_rn(zh, zh), zl, __fmaf_rn(zh, zh, -gh));
    const float kh = __fmul_rn(gh, ch);
    const float kl = __fadd_rn(__fmaf_rn(gh, ch, -kh), __fmaf_rn(gh, cl, __fmul_rn(gl, ch)));
    const float a = __fmaf_rn(zh, -0.5f, 1.0f);
    const float al = __fadd_rn(__fmaf_rn(zh, -0.5f, __fsub_rn(1.0f, a)), __fmul_rn(zl, -0.5f));
    r = __fadd_rn(a, kh);
    const float cosine = __fadd_rn(r, __fadd_rn(__fadd_rn(__fsub_rn(a, r), kh), __fadd_rn(al, kl)));

    const float c = quarter & 1u ? sine : cosine, s = quarter & 1u ? cosine : sine;
    return make_float2(quarter == 1u || quarter == 2u ? -c : c, quarter >= 2u ? -s : s);
}

__device__ __forceinline__ float2 rope_turn(const RopeView& r, int i, int pos)
{
    const float2 cs = rope_cos_sin(r.turns[i] * static_cast<unsigned long long>(static_cast<long long>(pos)));
    return make_float2(__fmul_rn(cs.x, r.magnitude), __fmul_rn(cs.y, r.magnitude));
}

// The two values of a pair, turned.
__device__ __forceinline__ float rope_first(float a, float b, float2 cs)
{
    return __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
}
__device__ __forceinline__ float rope_second(float a, float b, float2 cs)
{
    return __fadd_rn(__fmul_rn(a, cs.y), __fmul_rn(b, cs.x));
}

}  // namespace mmq
