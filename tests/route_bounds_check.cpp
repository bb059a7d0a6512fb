// Host check of the bounds within which routing by scores leaves an order to double
// precision (csrc/route_bounds.hpp): every fp32 operation is given its largest error, in
// the direction that moves two compared values apart the most, over grids of logits,
// biases and ranges; the bounds must hold what comes of it.  The errors, in u = 2^-24:
// an addition, product or division 1 of its result, the exponential 1.5 |x| + 2 (its
// argument in base 2 is rounded twice, the power is one last place off), the hardware's
// reciprocal 2.  Prints one line per check; exits nonzero if one does not hold.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <vector>

#include "route_bounds.hpp"

using namespace w4a4;

static const double u = std::ldexp(1.0, -24);
static int failures = 0;

static void holds(const char* what, double worst)
{
    std::printf("%s: %.4f of the bound\n", what, worst);
    if (!(worst <= 1.0)) ++failures;
}

// largest error of the sigmoid of l
static double sigmoid_error(double l)
{
    const double e = std::exp(-l), s = 1 / (1 + e), de = (1.5 * std::fabs(l) + 2) * u;
    const double up = 1 / ((1 + e * (1 - de)) * (1 - u)) * (1 + 2 * u), down = 1 / ((1 + e * (1 + de)) * (1 + u)) * (1 - 2 * u);
    return std::max(up - s, s - down);
}

static void check_sigmoid(bool sums, bool bias)
{
    double worst = 0;
    for (double top = -60; top <= 30; top += 0.05) {
        const double stop = 1 / (1 + std::exp(-top));
        double most = 0;
        for (double l = top; l > top - 20; l -= 0.05) most = std::max(most, sigmoid_error(l));
        for (double c : {0.0, 0.5, 1.0, 1.5, 4.0, 1000.0}) {   // choice values, in scores of the largest logit
            const double v = bias ? c * stop : 0, V = std::max(stop, v);
            // two values moved towards and past one another; a bias' sum rounds once more
            double apart = 2 * (most + (bias ? u * v : 0));
            if (sums) apart = 2 * apart + 2 * u * 2 * (bias ? v : stop);
            const float e = route_error(true, 16, (float)top, (float)V);
            worst = std::max(worst, apart / (sums ? route_sum_error(e, (float)V) : e));
        }
    }
    holds(sums ? bias ? "sigmoid, sums, bias" : "sigmoid, sums" : "sigmoid, bias", worst);
}

// n of E logits x below the largest, the others far below: all roundings in one direction
static void check_softmax(int lanes, int nv, bool sums, bool bias)
{
    double worst = 0;
    const int E = lanes * nv;
    for (int n = 0; n < E; n = n < 16 ? n + 1 : n * 2 - n / 2)
        for (double x = 0; x < 30; x += 0.05) {
            const double p = std::exp(-x), S = 1 + n * p;
            const double dp = (2.5 * x + 2) * u;   // (the argument's own rounding: |x| u of the power)
            const double additions = (nv - 1 + std::log2(lanes)) * u;
            const double dS = ((2 * u + n * p * dp) / S + additions);
            // scores of the largest and of the others
            const double s1 = 1 / S, d1 = 2.05 * u / S;   // e^-|y| (2.5 |y| + 2) is at most 2.05, for any logit
            const double common = dS + u;                 // of the reciprocal: the same for all scores
            for (double c : {0.0, 0.5, 1.0, 1.5, 4.0, 1000.0}) {
                const double v = bias ? c * s1 : 0, V = std::max(s1, v);
                // the scores that are compared lie between 0 and the largest
                double apart = 2 * (d1 + u * s1 + (bias ? u * v : 0)) + common * s1;
                if (sums) apart = 2 * apart + 2 * u * 2 * (bias ? v : s1);
                const float e = route_error(false, nv, 0.0f, (float)V);
                worst = std::max(worst, apart / (sums ? route_sum_error(e, (float)V) : e));
            }
        }
    char what[96];
    std::snprintf(what, sizeof what, "softmax of %d%s%s", E, sums ? ", sums" : "", bias ? ", bias" : "");
    holds(what, worst);
}

// y and the larger x, `error` apart, in fixed point: x's difference and product upward,
// y's downward, and the whole units of both up to one more apart
static void check_units(int bits)
{
    double worst = 0;
    for (double r : {1e-20, 1e-3, 1.0, 3.7, 1e20}) {
        const float unit = route_units(bits) / (float)r;
        for (double share = 1e-9; share < 0.3; share *= 1.07) {
            const float error = (float)(share * r);
            for (double at : {0.0, 0.1, 0.4999, 0.5, 0.7, 1.0}) {
                const double y = at * (r - error), x = y + error;
                const double units = x * (1 + u) * unit * (1 + u) - y * (1 - u) * unit * (1 - u) + 1;
                worst = std::max(worst, units / route_apart(bits, error, unit));
            }
        }
    }
    char what[64];
    std::snprintf(what, sizeof what, "units of %d bits", 32 - bits);
    holds(what, worst);
}

int main()
{
    check_sigmoid(false, true);
    check_sigmoid(true, false);
    check_sigmoid(true, true);
    for (int nv : {2, 4, 8, 16})
        for (int sums = 0; sums < 2; ++sums)
            for (int bias = 0; bias < 2; ++bias) check_softmax(16, nv, sums, bias);
    for (int nv : {4, 16})
        for (int sums = 0; sums < 2; ++sums)
            for (int bias = 0; bias < 2; ++bias) check_softmax(64, nv, sums, bias);
    for (int bits : {6, 8, 10}) check_units(bits);
    return failures ? 1 : 0;
}
