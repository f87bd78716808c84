// sample_weight.cuh — exp((x - max) / T) as a whole number of 2^-44, for
// spec_sample.  Host and device: its test compiles it without nvcc.
//
// Which tokens a row keeps, and which one is drawn, is decided where running sums
// of a vocabulary's weights pass a border.  Sums in 32 bits are off by 2^-22 or so,
// as much as a token's whole weight in a flat row, and depend on their order.  So a
// weight is made to about 2^-42 of itself, in pairs of floats (64-bit arithmetic
// has 1/64 of their rate here), and sums are of whole numbers: the same whatever
// their order, and exact.
#pragma once
#include <math.h>
#include <stdint.h>
#include <string.h>

#if defined(__CUDACC__)
#define SPECDEC_WEIGHT_FN __device__ __forceinline__
#define SPECDEC_WEIGHT_TABLE __device__ const
#else
#define SPECDEC_WEIGHT_FN inline
#define SPECDEC_WEIGHT_TABLE static const
#endif

namespace specdec {

constexpr int kWeightBits = 44;  // of the largest weight: 2^18 of them fit 64 bits
constexpr uint64_t kWeightOne = 1ull << kWeightBits;

#if defined(__CUDACC__)
__device__ __forceinline__ float w_add(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ float w_mul(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ float w_fma(float a, float b, float c) { return __fmaf_rn(a, b, c); }
__device__ __forceinline__ int32_t w_bits(float x) { return __float_as_int(x); }
__device__ __forceinline__ float w_float(int32_t x) { return __int_as_float(x); }
#else
inline float w_add(float a, float b) { return a + b; }  // (compiled without contraction)
inline float w_mul(float a, float b) { return a * b; }
inline float w_fma(float a, float b, float c) { return fmaf(a, b, c); }
inline int32_t w_bits(float x) {
  int32_t i;
  memcpy(&i, &x, 4);
  return i;
}
inline float w_float(int32_t x) {
  float f;
  memcpy(&f, &x, 4);
  return f;
}
#endif

// 2^(i / 256) as a float and what it leaves out (to 2^-49), from powers in 60
// decimal digits.
struct ExpPair {
  float hi, lo;
};
SPECDEC_WEIGHT_TABLE ExpPair kExp2Table[256] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.00b1b00000000p+0f, -0x1.6950d00000000p-26f}, {0x1.0163da0000000p+0f, 0x1.3f66660000000p-25f},
    {0x1.0216820000000p+0f, -0x1.789fb00000000p-25f}, {0x1.02c9a40000000p+0f, -0x1.887fa00000000p-28f}, {0x1.037d420000000p+0f, 0x1.c2377a0000000p-25f},
    {0x1.04315e0000000p+0f, 0x1.0dcff00000000p-25f}, {0x1.04e5f80000000p+0f, -0x1.a1356a0000000p-25f}, {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f},
    {0x1.0650a00000000p+0f, 0x1.c783f20000000p-25f}, {0x1.0706b20000000p+0f, 0x1.3bbedc0000000p-25f}, {0x1.07bd420000000p+0f, 0x1.6e55060000000p-25f},
    {0x1.0874520000000p+0f, -0x1.e2990e0000000p-26f}, {0x1.092be00000000p+0f, -0x1.333f040000000p-25f}, {0x1.09e3ec0000000p+0f, 0x1.58de700000000p-25f},
    {0x1.0a9c7a0000000p+0f, -0x1.3831ba0000000p-26f}, {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f}, {0x1.0c0f140000000p+0f, 0x1.791b220000000p-26f},
    {0x1.0cc9220000000p+0f, 0x1.6e48fe0000000p-25f}, {0x1.0d83b20000000p+0f, 0x1.9caef60000000p-27f}, {0x1.0e3ec40000000p+0f, -0x1.a585cc0000000p-25f},
    {0x1.0efa560000000p+0f, -0x1.02b1da0000000p-31f}, {0x1.0fb66a0000000p+0f, 0x1.ffda640000000p-25f}, {0x1.1073020000000p+0f, 0x1.1ae4680000000p-25f},
    {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f}, {0x1.11edba0000000p+0f, 0x1.6bc5560000000p-25f}, {0x1.12abdc0000000p+0f, 0x1.b0c7300000000p-30f},
    {0x1.136a820000000p+0f, -0x1.61bf6a0000000p-25f}, {0x1.1429aa0000000p+0f, 0x1.d525bc0000000p-25f}, {0x1.14e95a0000000p+0f, -0x1.9619da0000000p-25f},
    {0x1.15a98c0000000p+0f, 0x1.14b1ca0000000p-25f}, {0x1.166a460000000p+0f, -0x1.71c7880000000p-25f}, {0x1.172b840000000p+0f, -0x1.c157420000000p-27f},
    {0x1.17ed480000000p+0f, 0x1.a56ef00000000p-26f}, {0x1.18af940000000p+0f, -0x1.dcdc860000000p-26f}, {0x1.1972660000000p+0f, -0x1.f228b40000000p-26f},
    {0x1.1a35be0000000p+0f, 0x1.6df96e0000000p-25f}, {0x1.1af9a00000000p+0f, -0x1.fb1d780000000p-26f}, {0x1.1bbe080000000p+0f, 0x1.0117340000000p-26f},
    {0x1.1c82fa0000000p+0f, -0x1.5afc720000000p-25f}, {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f}, {0x1.1e0e760000000p+0f, -0x1.4bbfda0000000p-28f},
    {0x1.1ed5020000000p+0f, 0x1.7e6c8e0000000p-27f}, {0x1.1f9c180000000p+0f, 0x1.0e33940000000p-26f}, {0x1.2063b80000000p+0f, 0x1.0c519a0000000p-25f},
    {0x1.212be40000000p+0f, -0x1.50eafc0000000p-25f}, {0x1.21f49a0000000p+0f, -0x1.d0446e0000000p-25f}, {0x1.22bdda0000000p+0f, 0x1.3c89680000000p-27f},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.2452000000000p+0f, -0x1.1f7afe0000000p-26f}, {0x1.251ce40000000p+0f, 0x1.f654c80000000p-25f},
    {0x1.25e8580000000p+0f, -0x1.dc26320000000p-25f}, {0x1.26b4560000000p+0f, 0x1.789f380000000p-26f}, {0x1.2780e40000000p+0f, -0x1.7c441a0000000p-25f},
    {0x1.284dfe0000000p+0f, 0x1.f563800000000p-28f}, {0x1.291ba80000000p+0f, -0x1.4dc8920000000p-25f}, {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f},
    {0x1.2ab8a60000000p+0f, 0x1.b443c40000000p-26f}, {0x1.2b87fe0000000p+0f, -0x1.e4a4ce0000000p-25f}, {0x1.2c57e40000000p+0f, -0x1.a239340000000p-26f},
    {0x1.2d285a0000000p+0f, 0x1.b900c20000000p-26f}, {0x1.2df9620000000p+0f, -0x1.37d4ee0000000p-29f}, {0x1.2ecafa0000000p+0f, 0x1.27c5ea0000000p-25f},
    {0x1.2f9d240000000p+0f, 0x1.57b10e0000000p-25f}, {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f}, {0x1.31432e0000000p+0f, 0x1.bdd6600000000p-25f},
    {0x1.3217100000000p+0f, -0x1.d993e80000000p-27f}, {0x1.32eb840000000p+0f, -0x1.15c5740000000p-26f}, {0x1.33c08c0000000p+0f, -0x1.b37d200000000p-25f},
    {0x1.3496260000000p+0f, 0x1.b8fe8c0000000p-26f}, {0x1.356c560000000p+0f, -0x1.b5803c0000000p-30f}, {0x1.36431a0000000p+0f, 0x1.6f441e0000000p-27f},
    {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f}, {0x1.37f2620000000p+0f, 0x1.8f3aa40000000p-27f}, {0x1.38cae60000000p+0f, 0x1.a0bb0c0000000p-25f},
    {0x1.39a4020000000p+0f, -0x1.23afc40000000p-26f}, {0x1.3a7db40000000p+0f, -0x1.634c020000000p-25f}, {0x1.3b57fc0000000p+0f, -0x1.3930ba0000000p-32f},
    {0x1.3c32dc0000000p+0f, 0x1.89d4720000000p-27f}, {0x1.3d0e540000000p+0f, 0x1.3b785c0000000p-26f}, {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f},
    {0x1.3ec70e0000000p+0f, -0x1.c75d160000000p-29f}, {0x1.3fa4500000000p+0f, 0x1.2b20060000000p-26f}, {0x1.40822c0000000p+0f, 0x1.b3d0120000000p-27f},
    {0x1.4160a20000000p+0f, 0x1.f72e2a0000000p-28f}, {0x1.423fb20000000p+0f, 0x1.c251a20000000p-26f}, {0x1.431f5e0000000p+0f, -0x1.abd5da0000000p-26f},
    {0x1.43ffa40000000p+0f, -0x1.ed18b00000000p-30f}, {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f}, {0x1.45c2040000000p+0f, 0x1.53e9180000000p-27f},
    {0x1.46a41e0000000p+0f, 0x1.a3a00a0000000p-25f}, {0x1.4786d60000000p+0f, 0x1.a2cc8e0000000p-26f}, {0x1.486a2c0000000p+0f, -0x1.47d8660000000p-25f},
    {0x1.494e1e0000000p+0f, 0x1.92aed20000000p-28f}, {0x1.4a32b00000000p+0f, -0x1.e505840000000p-25f}, {0x1.4b17de0000000p+0f, 0x1.4db6fa0000000p-25f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.4ce41c0000000p+0f, -0x1.fa0fba0000000p-26f}, {0x1.4dcb2a0000000p+0f, -0x1.8088bc0000000p-26f},
    {0x1.4eb2d80000000p+0f, 0x1.d8abfe0000000p-28f}, {0x1.4f9b280000000p+0f, -0x1.2c5a6c0000000p-25f}, {0x1.5084180000000p+0f, -0x1.759c240000000p-29f},
    {0x1.516daa0000000p+0f, 0x1.67b3200000000p-27f}, {0x1.5257de0000000p+0f, 0x1.07e9de0000000p-25f}, {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f},
    {0x1.542e300000000p+0f, -0x1.612a5c0000000p-25f}, {0x1.551a4c0000000p+0f, 0x1.4bb2420000000p-25f}, {0x1.56070e0000000p+0f, -0x1.0b77980000000p-27f},
    {0x1.56f4740000000p+0f, -0x1.295b040000000p-25f}, {0x1.57e27e0000000p+0f, -0x1.074ecc0000000p-26f}, {0x1.58d12e0000000p+0f, -0x1.6d07000000000p-25f},
    {0x1.59c0820000000p+0f, 0x1.ffc1f20000000p-26f}, {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f}, {0x1.5ba1200000000p+0f, -0x1.15e1800000000p-26f},
    {0x1.5c92680000000p+0f, 0x1.4b28d60000000p-25f}, {0x1.5d845a0000000p+0f, -0x1.ecce8e0000000p-25f}, {0x1.5e76f20000000p+0f, -0x1.4a5bd60000000p-25f},
    {0x1.5f6a320000000p+0f, 0x1.b9d6e20000000p-29f}, {0x1.605e1c0000000p+0f, -0x1.a248fe0000000p-26f}, {0x1.6152ae0000000p+0f, 0x1.b37dbe0000000p-26f},
    {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f}, {0x1.633dd20000000p+0f, -0x1.736b020000000p-27f}, {0x1.6434640000000p+0f, -0x1.66679c0000000p-25f},
    {0x1.652ba00000000p+0f, -0x1.43704a0000000p-28f}, {0x1.6623880000000p+0f, 0x1.2a91120000000p-27f}, {0x1.671c1c0000000p+0f, 0x1.c20cfe0000000p-26f},
    {0x1.68155e0000000p+0f, -0x1.766ad20000000p-25f}, {0x1.690f4c0000000p+0f, -0x1.cc2d580000000p-25f}, {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f},
    {0x1.6b05300000000p+0f, -0x1.62ba300000000p-26f}, {0x1.6c01280000000p+0f, -0x1.5e84a80000000p-25f}, {0x1.6cfdce0000000p+0f, -0x1.15c4de0000000p-27f},
    {0x1.6dfb240000000p+0f, -0x1.cd72e80000000p-27f}, {0x1.6ef92a0000000p+0f, -0x1.e9b1460000000p-26f}, {0x1.6ff7e00000000p+0f, -0x1.ab9ae00000000p-26f},
    {0x1.70f7460000000p+0f, 0x1.bd0ba20000000p-26f}, {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f}, {0x1.72f8280000000p+0f, 0x1.bab4220000000p-26f},
    {0x1.73f9a40000000p+0f, 0x1.14b02e0000000p-25f}, {0x1.74fbd40000000p+0f, -0x1.4506800000000p-25f}, {0x1.75feb60000000p+0f, -0x1.37b3060000000p-25f},
    {0x1.77024c0000000p+0f, -0x1.ca923e0000000p-25f}, {0x1.7806940000000p+0f, 0x1.fbcba80000000p-25f}, {0x1.790b940000000p+0f, -0x1.d4f8c20000000p-26f},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.7b17b00000000p+0f, 0x1.2ed9fc0000000p-25f}, {0x1.7c1ed00000000p+0f, 0x1.30c1320000000p-28f},
    {0x1.7d26a60000000p+0f, 0x1.7fc3780000000p-27f}, {0x1.7e2f340000000p+0f, -0x1.2616340000000p-25f}, {0x1.7f38780000000p+0f, 0x1.2471240000000p-26f},
    {0x1.8042760000000p+0f, -0x1.783cbe0000000p-25f}, {0x1.814d2a0000000p+0f, 0x1.ba20dc0000000p-25f}, {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f},
    {0x1.8364c20000000p+0f, -0x1.46be080000000p-28f}, {0x1.8471a40000000p+0f, 0x1.88f1ec0000000p-26f}, {0x1.857f420000000p+0f, -0x1.0c149c0000000p-25f},
    {0x1.868d9a0000000p+0f, -0x1.2edb440000000p-26f}, {0x1.879cae0000000p+0f, -0x1.b396f20000000p-26f}, {0x1.88ac7e0000000p+0f, -0x1.9d665a0000000p-26f},
    {0x1.89bd0a0000000p+0f, 0x1.1e16040000000p-26f}, {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f}, {0x1.8be05c0000000p+0f, -0x1.4a7a220000000p-26f},
    {0x1.8cf3220000000p+0f, -0x1.29576e0000000p-25f}, {0x1.8e06a60000000p+0f, -0x1.f799280000000p-28f}, {0x1.8f1aea0000000p+0f, -0x1.baa2320000000p-26f},
    {0x1.902fee0000000p+0f, -0x1.fafa6e0000000p-25f}, {0x1.9145b00000000p+0f, 0x1.723ff80000000p-25f}, {0x1.925c360000000p+0f, -0x1.8aba040000000p-25f},
    {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f}, {0x1.948b820000000p+0f, 0x1.6bf31c0000000p-25f}, {0x1.95a44c0000000p+0f, 0x1.790a420000000p-25f},
    {0x1.96bdda0000000p+0f, -0x1.6263d40000000p-26f}, {0x1.97d82a0000000p+0f, -0x1.0d8d840000000p-31f}, {0x1.98f33e0000000p+0f, 0x1.1e88a80000000p-26f},
    {0x1.9a0f180000000p+0f, -0x1.e6bf080000000p-25f}, {0x1.9b2bb40000000p+0f, 0x1.aa7fc20000000p-25f}, {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f},
    {0x1.9d67420000000p+0f, -0x1.ad11ca0000000p-26f}, {0x1.9e86320000000p+0f, -0x1.8737380000000p-26f}, {0x1.9fa5e80000000p+0f, 0x1.a0fe540000000p-25f},
    {0x1.a0c6680000000p+0f, -0x1.2886a60000000p-26f}, {0x1.a1e7ae0000000p+0f, 0x1.b1d7180000000p-25f}, {0x1.a309be0000000p+0f, 0x1.8945a60000000p-25f},
    {0x1.a42c980000000p+0f, 0x1.182b5e0000000p-30f}, {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f}, {0x1.a674a80000000p+0f, 0x1.5e8c0a0000000p-25f},
    {0x1.a799e20000000p+0f, -0x1.99e9940000000p-25f}, {0x1.a8bfe60000000p+0f, -0x1.87da340000000p-25f}, {0x1.a9e6b60000000p+0f, -0x1.50c0480000000p-25f},
    {0x1.ab0e520000000p+0f, 0x1.356eba0000000p-28f}, {0x1.ac36bc0000000p+0f, -0x1.6064320000000p-31f}, {0x1.ad5ff40000000p+0f, -0x1.70f6220000000p-26f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.afb4ce0000000p+0f, 0x1.88bcc00000000p-26f}, {0x1.b0e0720000000p+0f, 0x1.31b6cc0000000p-25f},
    {0x1.b20ce60000000p+0f, 0x1.93512a0000000p-25f}, {0x1.b33a2c0000000p+0f, -0x1.ec3a820000000p-26f}, {0x1.b468420000000p+0f, -0x1.4916ca0000000p-25f},
    {0x1.b597280000000p+0f, 0x1.bcab280000000p-25f}, {0x1.b6c6e20000000p+0f, 0x1.3e38a60000000p-25f}, {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f},
    {0x1.b928d00000000p+0f, -0x1.bb16c40000000p-25f}, {0x1.ba5b040000000p+0f, -0x1.ebdf360000000p-25f}, {0x1.bb8e0c0000000p+0f, -0x1.0cb21c0000000p-25f},
    {0x1.bcc1ea0000000p+0f, -0x1.f687c60000000p-25f}, {0x1.bdf69c0000000p+0f, 0x1.f9d1040000000p-27f}, {0x1.bf2c260000000p+0f, -0x1.0a387e0000000p-26f},
    {0x1.c062860000000p+0f, 0x1.41b33c0000000p-28f}, {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f}, {0x1.c2d1ce0000000p+0f, -0x1.8166b60000000p-26f},
    {0x1.c40ab60000000p+0f, -0x1.7c2c980000000p-39f}, {0x1.c544780000000p+0f, -0x1.c141380000000p-26f}, {0x1.c67f120000000p+0f, 0x1.cafa2a0000000p-25f},
    {0x1.c7ba880000000p+0f, 0x1.3119260000000p-25f}, {0x1.c8f6da0000000p+0f, -0x1.7f230a0000000p-25f}, {0x1.ca34060000000p+0f, -0x1.15c7640000000p-25f},
    {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f}, {0x1.ccb0f20000000p+0f, 0x1.cda2ce0000000p-25f}, {0x1.cdf0b60000000p+0f, -0x1.5447800000000p-25f},
    {0x1.cf31560000000p+0f, -0x1.2915240000000p-26f}, {0x1.d072d40000000p+0f, 0x1.40f1300000000p-25f}, {0x1.d1b5320000000p+0f, 0x1.61192e0000000p-25f},
    {0x1.d2f8700000000p+0f, 0x1.01b13e0000000p-25f}, {0x1.d43c8e0000000p+0f, 0x1.59543a0000000p-25f}, {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f},
    {0x1.d6c76e0000000p+0f, 0x1.0c5cda0000000p-25f}, {0x1.d80e320000000p+0f, -0x1.26cf8e0000000p-25f}, {0x1.d955d80000000p+0f, -0x1.c013f20000000p-25f},
    {0x1.da9e600000000p+0f, 0x1.ed99420000000p-27f}, {0x1.dbe7ce0000000p+0f, -0x1.38af9e0000000p-25f}, {0x1.dd32200000000p+0f, -0x1.9fc9740000000p-25f},
    {0x1.de7d560000000p+0f, 0x1.0701960000000p-26f}, {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f}, {0x1.e116760000000p+0f, 0x1.632fa20000000p-25f},
    {0x1.e264620000000p+0f, -0x1.614bda0000000p-25f}, {0x1.e3b3340000000p+0f, -0x1.3a447c0000000p-26f}, {0x1.e502ee0000000p+0f, 0x1.e2cffe0000000p-26f},
    {0x1.e653920000000p+0f, 0x1.19db5e0000000p-26f}, {0x1.e7a5200000000p+0f, -0x1.0e2ce00000000p-26f}, {0x1.e8f7980000000p+0f, -0x1.0649180000000p-25f},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.eb9f480000000p+0f, 0x1.9f329c0000000p-26f}, {0x1.ecf4820000000p+0f, 0x1.b1ccfe0000000p-25f},
    {0x1.ee4aaa0000000p+0f, 0x1.0c42880000000p-27f}, {0x1.efa1be0000000p+0f, 0x1.cc2b440000000p-25f}, {0x1.f0f9c20000000p+0f, -0x1.a4df6c0000000p-27f},
    {0x1.f252b40000000p+0f, -0x1.1288ae0000000p-25f}, {0x1.f3ac940000000p+0f, 0x1.1bae4e0000000p-25f}, {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f},
    {0x1.f663280000000p+0f, -0x1.9deec20000000p-26f}, {0x1.f7bfda0000000p+0f, 0x1.b397c20000000p-25f}, {0x1.f91d800000000p+0f, 0x1.121e440000000p-27f},
    {0x1.fa7c180000000p+0f, 0x1.9e90d80000000p-28f}, {0x1.fbdba40000000p+0f, -0x1.2da55e0000000p-25f}, {0x1.fd3c220000000p+0f, 0x1.71ee3e0000000p-25f},
    {0x1.fe9d960000000p+0f, 0x1.65447c0000000p-25f},
};

// log2(e) / T in two floats.
struct WeightScale {
  float hi, lo;
};

// x <= max, both finite.  With t = (x - max) log2(e) / T = k + i / 256 + r,
// |r| <= 2^-9, the weight is 2^k 2^(i / 256) e^(r ln 2).  A weight below 2^-45
// is 0.
SPECDEC_WEIGHT_FN uint64_t sample_weight(float x, float max, WeightScale s, const ExpPair* table) {
  // x - max and the rest that it leaves, exactly
  const float d = w_add(x, -max), back = w_add(d, -x);
  const float rest = w_add(w_add(x, -w_add(d, -back)), -w_add(max, back));
  const float t = w_mul(d, s.hi);
  if (!(t > -48.f)) return 0;
  float tl = w_fma(d, s.hi, -t);
  tl = w_fma(d, s.lo, tl);
  tl = w_fma(rest, s.hi, tl);
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to whole numbers
  const float z = w_fma(t, 256.f, kMagic);
  const int32_t n = w_bits(z) - 0x4B400000;
  const float r = w_fma(w_add(z, -kMagic), -1.f / 256.f, t);  // exact
  const ExpPair p = table[n & 255];
  // e^(r ln 2) - 1: ln 2 in two floats for the first power, one for the others
  constexpr float kL1 = 0x1.62e430p-1f, kL1Rest = -0x1.05c610p-29f;
  constexpr float kL2 = 0x1.ebfbe0p-3f, kL3 = 0x1.c6b08ep-5f, kL4 = 0x1.3b2ab6p-7f;
  const float a = w_mul(r, kL1);
  float al = w_fma(r, kL1, -a);
  al = w_fma(r, kL1Rest, al);
  al = w_fma(tl, kL1, al);
  const float rr = w_add(r, tl);
  al = w_fma(w_mul(rr, rr), w_fma(rr, w_fma(rr, kL4, kL3), kL2), al);
  // times the table's pair, less its first
  const float b = w_mul(p.hi, a);
  float bl = w_fma(p.hi, a, -b);
  bl = w_fma(p.hi, al, bl);
  bl = w_fma(p.lo, a, bl);
  bl = w_add(bl, p.lo);
  // times 2^k (at most 1 in all), in whole numbers of 2^-22 and 2^-44
  const float k = w_float(((n >> 8) + 127) << 23), hi = w_mul(p.hi, k), lo = w_mul(w_add(b, bl), k);
  const float left = w_mul(w_add(w_add(b, -w_add(b, bl)), bl), k);
  const float v = w_add(hi, lo), rest2 = w_add(w_add(w_add(hi, -v), lo), left);
  constexpr float kMagic22 = 3.f, kMagic44 = 1.5f * 0x1p-21f;
  const float v1 = w_add(v, kMagic22);
  const float v2 = w_add(w_add(w_add(v, -w_add(v1, -kMagic22)), rest2), kMagic44);
  return static_cast<uint64_t>(static_cast<int64_t>(w_bits(v1) - w_bits(kMagic22)) * (1 << 22) + (w_bits(v2) - w_bits(kMagic44)));
}

}  // namespace specdec
