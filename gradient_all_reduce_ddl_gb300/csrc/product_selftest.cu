// product_selftest.cu -- the product kernels with stops that make their waits run
// out (internal; the wait self-tests of include/ddl.h).
#define DDL_PRODUCT_SELFTEST 1
#include "product_kernels.cu"
